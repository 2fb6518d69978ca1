// Gated linear recurrence, one state a channel: parameters, the gates, and the carry between chunks.
//
//   l = -rate softplus(decay) sr, sr = sigmoid(r + rb);  a = exp(l);  e = sqrt(1 - a^2)
//   h[t] = a h[t-1] + e si x, si = sigmoid(i + ib);  out = h silu(z)
//   backward: dh = dout silu(z);  g[t] = dh + a[t+1] g[t+1];  W = l a g h[t-1] - (l / e) a^2 g si x
//             dx = g e si;  di = g e x si (1 - si);  dr = (1 - sr) W;  ddecay = sigmoid(decay) / softplus(decay) sum W
//
// A step maps h to a h + b, and steps join: (a, b) then (a', b') is (a' a, a' b + b'). So tokens are walked in pieces: a lane
// owns VC neighbouring channels, a wave TT neighbouring tokens, which it keeps in registers as (a, b); the waves' joined steps
// meet in LDS, where each wave finds the state that enters its tokens.
#pragma once
#include "layer.hpp"

namespace mimo {
namespace layer {

struct RecurParams {
    Seqs q;
    int D, nvec, has_z, zero_tail, chunked;
    unsigned tiles;                 // blocks along the channels
    float rate;
    Rows x, r, i, z, dout;
    const float *decay, *rb, *ib;
    const float *init, *dstate;
    void* out;
    float* state;
    float *agg_h, *agg_p, *agg_g;   // [slots][D]: a chunk's last state from zero, its product of a, the adjoint that leaves it to the left
    // backward
    void *dx, *dr, *di, *dz;
    float *ddecay, *drb, *dib, *dinit;
    float* part;                    // [slots][3][D]
    long slots;
};

// first row of the flat token axis of a place
__device__ __forceinline__ long recur_row(const Seqs& q, const Place& pl) { return q.cu ? (long)pl.row0 : (long)pl.i * q.S; }

// a = 2^l2 and 1 - a^2. Near a = 1 the difference would leave few bits (and e, of which tokens a slow channel takes in little,
// with them): there the series of -expm1(y), y = 2 ln a, to y^6 (its next term is below 2^-25 of the sum for |y| < 1/4); elsewhere
// one rounding, and a's error, which the difference enlarges five times at most.
__device__ __forceinline__ void keep_and_enter(float l2, float& a, float& e2) {
    a = exp2_hw(l2);
    const float y = l2 * (2.f * LN2);
    float s = __builtin_fmaf(y, 1.f / 720.f, 1.f / 120.f);
    s = __builtin_fmaf(y, s, 1.f / 24.f);
    s = __builtin_fmaf(y, s, 1.f / 6.f);
    s = __builtin_fmaf(y, s, 0.5f);
    s = __builtin_fmaf(y, s, 1.f);
    e2 = y > -0.25f ? -y * s : __builtin_fmaf(-a, a, 1.f);
}
__device__ __forceinline__ float root(float x) { return __builtin_amdgcn_sqrtf(x); }

// a lane's parameters: -rate softplus(decay) log2(e), and the biases
template <int VC> struct Gates {
    float speed[VC], rb[VC], ib[VC];
    __device__ __forceinline__ Gates(const RecurParams& p, unsigned d) {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            speed[v] = -p.rate * LOG2E * softplus(p.decay[d + v]);
            rb[v] = p.rb ? p.rb[d + v] : 0.f;
            ib[v] = p.ib ? p.ib[d + v] : 0.f;
        }
    }
};

// TT rows from t0 on (the last one again where they end before), at a scalar base and a lane's offset
template <int DT, int VC, int TT> struct RowsOf {
    Pack<DT, VC> t[TT];
    __device__ __forceinline__ void fetch(const raw_t<DT>* base, long ts, int t0, int last, unsigned d) {
#pragma unroll
        for (int k = 0; k < TT; ++k) t[k] = load<DT, VC>(base + min(t0 + k, last) * ts + d);
    }
};

// The states that enter the chunks of sequence blockIdx.z, in place of the aggregates. Wave w of a block takes SPAN chunks of
// every SPAN * waves: it folds them from zero, the waves' folds are chained in LDS, and it walks them again from what enters
// them, so that all loads of up to 128 chunks are in flight together. With ADJ, blockIdx.y = 1 runs the adjoints from the last
// chunk to the first, from dstate, and leaves the gradient of the initial state.
constexpr int RSPAN = 8, RSPAN_WAVES = 16;
template <bool ADJ> __global__ __launch_bounds__(64 * RSPAN_WAVES) void k_recur_carry(RecurParams p) {
    __shared__ float s_h[RSPAN_WAVES][64], s_p[RSPAN_WAVES][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int i = blockIdx.z;
    const unsigned d0 = blockIdx.x * 64 + lane;
    const bool rev = ADJ && blockIdx.y, act = d0 < (unsigned)p.D;
    const unsigned d = act ? d0 : 0;
    const long D = p.D;
    const int slot0 = p.q.cu ? p.q.base(i) : i * p.q.nc;
    const int len = p.q.cu ? max((i < p.q.n ? p.q.start(i + 1) : p.q.S) - p.q.start(i), 0) : p.q.S;
    const int nc = max((len + p.q.CH - 1) / p.q.CH, 1);
    const int have = ADJ ? (len > 0 ? nc : 0) : nc - 1;    // chunks with an aggregate: the forward pass needs none of the last
    const float* from = rev ? p.dstate : p.init;
    float h = from ? from[(long)i * D + d] : 0.f;
    float* agg = (rev ? p.agg_g : p.agg_h) + (long)slot0 * D + d;
    const float* prod = p.agg_p + (long)slot0 * D + d;
    for (int j0 = 0; j0 < nc; j0 += RSPAN * waves) {
        float x[RSPAN], e[RSPAN], fold = 0.f, all = 1.f;
#pragma unroll
        for (int k = 0; k < RSPAN; ++k) {
            const int j = j0 + w * RSPAN + k, at = rev ? nc - 1 - j : j;
            x[k] = j < have ? agg[(long)at * D] : 0.f;
            e[k] = j < have ? prod[(long)at * D] : 1.f;
        }
#pragma unroll
        for (int k = 0; k < RSPAN; ++k) {
            fold = __builtin_fmaf(e[k], fold, x[k]);
            all *= e[k];
        }
        s_h[w][lane] = fold;
        s_p[w][lane] = all;
        __syncthreads();
        float g = h;
        for (int o = 0; o < waves; ++o) {
            if (o == w) g = h;
            h = __builtin_fmaf(s_p[o][lane], h, s_h[o][lane]);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < RSPAN; ++k) {
            const int j = j0 + w * RSPAN + k;
            if (j < nc && act) agg[(long)(rev ? nc - 1 - j : j) * D] = g;
            g = __builtin_fmaf(e[k], g, x[k]);
        }
    }
    if (rev && p.dinit && w == 0 && act) p.dinit[(long)i * D + d] = h;
}

// ---------------------------------------------------------------- host side
// Waves for the chunks of a sequence, of a packed one for twice the average: longer ones take more rounds.
template <bool ADJ> mimo_status launch_recur_carry(const RecurParams& p, hipStream_t st) {
    long chunks = p.q.nc;
    if (p.q.cu && 2 * p.slots / p.q.n < chunks) chunks = 2 * p.slots / p.q.n;
    const int waves = (int)(chunks <= RSPAN ? 1 : chunks < RSPAN * RSPAN_WAVES ? (chunks + RSPAN - 1) / RSPAN : RSPAN_WAVES);
    return launch(&k_recur_carry<ADJ>, dim3((unsigned)((p.D + 63) / 64), ADJ ? 2 : 1, p.q.n), 64 * waves, 0, st, p);
}
inline mimo_status check_recur(int64_t n, int64_t S, int64_t D, int dtype, float rate) {
    const mimo_status s = check_sequences(n, S, D, dtype);
    if (s != MIMO_OK) return s;
    if (!(rate >= 0.f) || rate > 3e38f) return bad("rate must be finite and not negative");
    if (n * S > (int64_t)1 << 40) return unsupported("too many tokens");
    return MIMO_OK;
}
// the data of a call: two channels a lane where all of it allows
inline int channels_of(int64_t D, int dtype, bool packed, std::initializer_list<const mamba_rows*> rows, std::initializer_list<const void*> dense) {
    const int esz = dtype == F32 ? 4 : 2;
    bool two = D % 2 == 0;
    for (const mamba_rows* r : rows) two = two && (!r->data || aligned(r->data, packed ? 0 : r->batch_stride, r->token_stride, 2 * esz, esz));
    for (const void* x : dense) two = two && aligned(x, 0, 0, 2 * esz, 1);
    return two ? 2 : 1;
}

}  // namespace layer
}  // namespace mimo
