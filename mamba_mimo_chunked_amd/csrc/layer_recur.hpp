// Gated linear recurrence, one state a channel: parameters, the gates, and rows of tokens.
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
#include <initializer_list>

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
    // forward: what chunks tell those behind them, [slots and groups][D], and the chunks taken of each tile
    unsigned long long* told;
    unsigned* taken;
    long words;
    // backward
    float *agg_h, *agg_p, *agg_g;   // [slots][D]: a chunk's last state from zero, its product of a, the adjoint that leaves it to the left
    void *dx, *dr, *di, *dz;
    float *ddecay, *drb, *dib, *dinit;
    float* part;                    // [slots][3][D]
    long slots;
};

// place(), by a whole wave: its lanes look at 64 sequences at a time, two or three dependent loads where bisection takes up to
// sixteen, which is what blocks of short sequences wait for (2000 sequences of 8 tokens, D = 2048, forward: 795 us, 990 by bisection).
__device__ __forceinline__ Place place_by_wave(const Seqs& q, int slot) {
    if (q.cu == nullptr) return place(q, slot);
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = q.n;           // the largest sequence whose base(lo) <= slot is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
        // those in front of the first that is behind: base(lo) <= slot, also where cu_seqlens decrease
        const unsigned long long behind = ~__ballot(at <= hi && q.base(min(at, hi)) <= slot);
        const int below = behind ? __builtin_ctzll(behind) : 64;
        const int from = lo + below * step;
        hi = min(hi, from + step - 1);
        lo = from;
    }
    Place r;
    r.i = lo;
    r.j = slot - q.base(lo);
    r.row0 = q.start(lo);
    r.len = max((lo < q.n ? q.start(lo + 1) : q.S) - r.row0, 0);
    r.ok = r.j == 0 || (long)r.j * q.CH < r.len;
    return r;
}

// first row of the flat token axis of a place
__device__ __forceinline__ long recur_row(const Seqs& q, const Place& pl) { return q.cu ? (long)pl.row0 : (long)pl.i * q.S; }

// a = 2^l2 and 1 - a^2. Near a = 1 the difference would leave few bits (and e, of which tokens a slow channel takes in little,
// with them): there the series of -expm1(y), y = 2 ln a, to y^6 (its next term is below 2^-24 of the sum for |y| < 1/4); elsewhere
// one rounding, and a's error, which the difference enlarges 2 a^2 / (1 - a^2) times, some seven at most.
__device__ __forceinline__ void keep_and_enter(float l2, float& a, float& e2) {
    a = exp2_hw(l2);
    const float y = l2 * (2.f * LN2);
    float s = __builtin_fmaf(y, 1.f / 720.f, 1.f / 120.f);
    s = __builtin_fmaf(y, s, 1.f / 24.f);
    s = __builtin_fmaf(y, s, 1.f / 6.f);
    s = __builtin_fmaf(y, s, 0.5f);
    s = -y * __builtin_fmaf(y, s, 1.f);
    asm("" : "+v"(s));      // both are computed: a branch for each value costs more than the series
    e2 = y > -0.25f ? s : __builtin_fmaf(-a, a, 1.f);
}
__device__ __forceinline__ float root(float x) { return __builtin_amdgcn_sqrtf(x); }

// From here on a step keeps nothing, and l itself stays in range.
constexpr float FASTEST = 1e30f;
// Below it a channel counts as one that forgets nothing: what enters it in a token is below 2e-19 of x, and from 2e-39 down ln(2) / speed is infinite.
constexpr float SLOWEST = 0x1p-126f;
// a lane's parameters: -rate softplus(decay) log2(e), and the biases times -log2(e)
template <int VC> struct Gates {
    float speed[VC], rb[VC], ib[VC];
    // sigmoid(x + bias), in one multiply-add, 2^x, an addition and a reciprocal
    __device__ __forceinline__ static float open(float x, float bias) {
        return __builtin_amdgcn_rcpf(1.f + exp2_hw(__builtin_fmaf(x, -LOG2E, bias)));
    }
    __device__ __forceinline__ Gates(const RecurParams& p, unsigned d) {
#pragma unroll
        for (int v = 0; v < VC; ++v) {
            const float s = LOG2E * (p.rate * softplus(p.decay[d + v]));     // in this order: LOG2E * softplus may be infinite, and a rate zero
            speed[v] = s > FASTEST ? -FASTEST : s < SLOWEST ? 0.f : -s;
            rb[v] = p.rb ? -LOG2E * p.rb[d + v] : 0.f;
            ib[v] = p.ib ? -LOG2E * p.ib[d + v] : 0.f;
        }
    }
};

// Rows of a tile of tokens as a buffer: a lane's offset in bytes (vector), a row's (scalar, 32 bits: MAMBA_RECUR_MAX_STRIDE) and the
// tile's base. With pointers the compiler adds 64-bit addresses in vector registers and computes those of all rows first, spilling
// scalar registers over it; so, too, the barriers beside an access. Loads from the buffer's end on give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, unsigned bytes = ~0u) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x27000);
}
// AUX: the access's cache policy, NT for data that passes by
constexpr int NT = 2;
template <int DT, int VC, int AUX = 0> __device__ __forceinline__ Pack<DT, VC> load_at(__amdgpu_buffer_rsrc_t buf, unsigned lane, unsigned row) {
    typedef Pack<DT, VC> Raw;
    if constexpr (sizeof(Raw) == 2) return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b16(buf, lane, row, AUX));
    else return __builtin_bit_cast(Raw, __builtin_amdgcn_raw_buffer_load_b32(buf, lane, row, AUX));
}
template <int DT, int VC, int AUX = 0> __device__ __forceinline__ void store_at(__amdgpu_buffer_rsrc_t buf, unsigned lane, unsigned row, const float (&x)[VC]) {
    typedef Pack<DT, VC> Raw;
    Raw o;
    if constexpr (DT == BF16 && VC == 2) o = __builtin_bit_cast(Raw, __builtin_convertvector(f2{x[0], x[1]}, b16x2));
    else {
#pragma unroll
        for (int v = 0; v < VC; ++v) o.v[v] = to_raw<DT>(x[v]);
    }
    if constexpr (sizeof(Raw) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, o), buf, lane, row, AUX);
    else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, o), buf, lane, row, AUX);
}
// the same value, of which the compiler knows nothing
template <int DT, int VC> __device__ __forceinline__ void renew(Pack<DT, VC>& x) {
    typedef Pack<DT, VC> Raw;
    if constexpr (sizeof(Raw) == 2) {
        unsigned r = __builtin_bit_cast(unsigned short, x);
        asm("" : "+v"(r));
        x = __builtin_bit_cast(Raw, (unsigned short)r);
    } else {
        unsigned r = __builtin_bit_cast(unsigned, x);
        asm("" : "+v"(r));
        x = __builtin_bit_cast(Raw, r);
    }
}
// One stream's rows of a wave's tokens, TT from t0 on, asked for one by one, so that streams can be asked for token by token and a
// token's work starts when its own rows are there. Rows from t1 on are zeros: they are asked for at the buffer's end, so nothing is read
// where t1 <= t0.
template <int DT, int VC, int TT, int AUX = 0> struct RowsOf {
    Pack<DT, VC> t[TT];
    unsigned step, at, end;
    int left;
    __amdgpu_buffer_rsrc_t rows;
    __device__ __forceinline__ void place(const Rows& r, const Place& pl, int D, int t0, int t1) {
        step = (unsigned)r.ts * sizeof(raw_t<DT>), at = 0;
        end = (unsigned)(min(max(t1 - t0, 1), TT) - 1) * step + D * sizeof(raw_t<DT>);
        left = t1 - t0;
        asm("" : "+s"(left));       // conditions of its own: those that streams share would fill the scalar registers
        rows = buffer_of(layer::at<DT>(r, pl) + t0 * r.ts, end);
    }
    __device__ __forceinline__ void fetch(int k, unsigned lane) {
        t[k] = load_at<DT, VC, AUX>(rows, lane, k < left ? at : end);
        at += step;
        __builtin_amdgcn_sched_barrier(0);
    }
};
// the exponent's factor for token k: none behind the chunk, whose a is one and which nothing enters
template <int VC> __device__ __forceinline__ float speed_of(const Gates<VC>& gates, int v, int k, int left) { return k < left ? gates.speed[v] : 0.f; }

// ---------------------------------------------------------------- host side
inline mimo_status check_recur(int64_t n, int64_t S, int64_t D, int dtype, float rate) {
    const mimo_status s = check_sequences(n, S, D, dtype);
    if (s != MIMO_OK) return s;
    if (!(rate >= 0.f) || rate > 3e38f) return bad("rate must be finite and not negative");
    if (n * S > (int64_t)1 << 40) return unsupported("too many tokens");
    return MIMO_OK;
}
// the rows of a tile of tokens lie within 32 bits of its first; a single token's stride is not used
inline mimo_status check_strides(int64_t S, std::initializer_list<const mamba_rows*> rows) {
    if (S == 1) return MIMO_OK;
    for (const mamba_rows* r : rows)
        if (r->data && (r->token_stride < 0 || r->token_stride > MAMBA_RECUR_MAX_STRIDE)) return unsupported("token strides beyond 2^26 elements");
    return MIMO_OK;
}
// Whether a call of so many streams passes the last-level cache by: it is larger than it, 256 MB, and its rows are whole lines of 128 bytes
// (parts of lines that nothing keeps are fetched again: [16384, 1001] backward, bf16, 194 us past the cache, 164 through it, fp32 266 and 253).
template <int DT> bool passes_by(const Seqs& q, int D, int streams) {
    const long row = (long)D * sizeof(raw_t<DT>);
    return row % 128 == 0 && (q.cu ? (long)q.S : (long)q.n * q.S) * row * streams > 256L << 20;
}
// Waves of a block of TT tokens each, and with them the tokens of a chunk. The last chunk of a packed sequence leaves some of them idle, so
// there are fewer, and fewest where the sequences have less than 64 tokens in the mean; short dense sequences have one chunk that fits.
// bf16, 16000 tokens, D = 2048, in us with 8, 4 and 2:
//   mean length     8               32              100             200             400             dense [1 x 8192]
//   forward     555 312 203     192 131 110     120  97  97     104  91  97      94  88  96      47  47  61
//   backward    877 547 418     372 283 257     260 225 227     234 217 222     215 206 219     102 109 118
// The mean counts empty sequences too, which a batch that is padded to a fixed number of them has. The same tokens in 8 long sequences
// (forward, backward; one long sequence): 8 in all 83, 201 (82, 208); 250, the last by 4 waves, 95, 222 (92, 273); 251, by 2, 99, 228 (110,
// 280); 2000 153, 351 (164, 414): a chunk's place for each empty sequence costs more than the waves that its mean brings.
inline int waves_of(bool packed, int64_t n, int64_t S, int TT) {
    if (packed) return S / n < 64 ? 2 : 4;
    return S <= 2 * TT ? 2 : S <= 4 * TT ? 4 : 8;
}
// channels of a lane: four bytes of them where all data allows
inline int channels_of(int64_t D, int dtype, bool packed, std::initializer_list<const mamba_rows*> rows, std::initializer_list<const void*> dense) {
    bool two = dtype != F32 && D % 2 == 0;
    for (const mamba_rows* r : rows) two = two && (!r->data || aligned(r->data, packed ? 0 : r->batch_stride, r->token_stride, 4, 2));
    for (const void* x : dense) two = two && aligned(x, 0, 0, 4, 1);
    return two ? 2 : 1;
}

}  // namespace layer
}  // namespace mimo
