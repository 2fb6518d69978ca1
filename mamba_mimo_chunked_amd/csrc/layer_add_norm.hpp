// Addition to the residual stream and root-mean-square norm of the sum: what the forward and the backward pass share.
//
//   v = dropout(x) + residual;  r = 1 / sqrt(mean(v^2) + eps);  y = v r w
//   backward: q = dout w;  hat = v r;  dv = r (q - hat mean(q hat)) + dsum;  dw = sum dout hat;  dx = dropout(dv)
//
// A row belongs to TPR = 8, 16, 32, 64 or 128 lanes, or (TPR = 0) to the whole block, of up to 16 waves; thread t takes the eight columns from 8 t
// on (and, in rows beyond 8192 columns, 8 threads further on), whatever the types: 16 bytes of a 16-bit type, twice 16 of fp32, 8 of an 8-bit
// output, and the eight elements that one counter of the generator covers. A row has as few lanes as it needs, as idle ones cost as much as
// others. bf16, 16.8 M elements, backward, us: 64 columns by 8 lanes 29.5, by 16 41.3; 256 by 32 29.2, by 64 42.9; 2056 by 5 waves 34.5, by 8
// 45.3; 4104 by 9 waves 32.2, by 16 57. Rows of two waves are two to a block ([16384, 1000]: 30.3, one by one 34.8).
#pragma once
#include "layer.hpp"

namespace mimo {
namespace layer {

constexpr int NV = 8;   // columns of a thread's access

template <int TPR> __device__ __forceinline__ int lane_of_row() { return TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x; }
template <int TPR> __device__ __forceinline__ int lanes_of_row() { return TPR ? TPR : blockDim.x; }
// the sum over the threads of a row, in all of them; `s`: LDS of a float a wave, safe to use again after the
// next call on another one
template <int TPR> __device__ __forceinline__ float sum_row(float x, float* s) {
    if constexpr (TPR && TPR <= 64) return sum_wave<TPR>(x);
    else {
        x = sum_wave<64>(x);
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
        __syncthreads();
        const unsigned k = threadIdx.x & 15;
        if constexpr (TPR) return s[threadIdx.x >> 7 << 1] + s[(threadIdx.x >> 7 << 1) + 1];
        else return sum_wave<16>(k < blockDim.x >> 6 ? s[k] : 0.f);
    }
}
constexpr int most_threads(int TPR) { return TPR ? 256 : 1024; }

// Eight neighbouring elements from column c of a row of D on, zeros behind the row. WIDE: rows of whole, aligned 16-byte accesses.
// Else accesses of 16 bytes at any element's address, which global memory takes; the row's last, broken eight are read as the
// row's last eight elements and moved into place when they are used, so that no lane reads otherwise than its neighbours ([8192, 2047]
// bf16 with a stream in fp32 and dropout, forward: 42 us, 123 with single elements).
template <class V, int ESZ> struct Loose { typedef V __attribute__((aligned(ESZ))) type; };
typedef unsigned quad __attribute__((ext_vector_type(4)));
template <int DT, bool WIDE> struct Eight {
    typedef raw_t<DT> raw;
    static constexpr int V = 16 / sizeof(raw);
    typedef Pack<DT, V> Raw;
    Raw t[NV / V];
    __device__ __forceinline__ void fetch(const raw* p, int c, int D) {
        if (WIDE || D >= NV) {
            if (c >= D) return;
            p += WIDE ? c : min(c, D - NV);
#pragma unroll
            for (int k = 0; k < NV / V; ++k) {
                if constexpr (WIDE) t[k] = load<DT, V>(p + V * k);
                else t[k] = __builtin_bit_cast(Raw, (quad)*reinterpret_cast<const typename Loose<quad, sizeof(raw)>::type*>(p + V * k));
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) t[k / V].v[k % V] = c + k < D ? p[c + k] : raw(0);
        }
    }
    __device__ __forceinline__ void read(int c, int D, float (&x)[NV]) const {
#pragma unroll
        for (int k = 0; k < NV; ++k) x[k] = c < D ? to_f<DT>(t[k / V].v[k % V]) : 0.f;
        if (!WIDE && c < D && c + NV > D && D >= NV) {
            const int by = c + NV - D;
#pragma unroll
            for (int s = 4; s > 0; s /= 2)
#pragma unroll
                for (int k = 0; k < NV; ++k) x[k] = by & s ? (k + s < NV ? x[k + s] : 0.f) : x[k];
        }
    }
};
template <int DT, bool WIDE> __device__ __forceinline__ void put8(raw_t<DT>* p, int c, int D, const float (&x)[NV]) {
    typedef raw_t<DT> raw;
    constexpr int V = 16 / sizeof(raw);
    if (WIDE ? c < D : c + NV <= D) {
#pragma unroll
        for (int k = 0; k < NV / V; ++k) {
            Pack<DT, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = to_raw<DT>(x[k * V + i]);
            if constexpr (WIDE) *reinterpret_cast<Pack<DT, V>*>(p + c + V * k) = o;
            else *reinterpret_cast<typename Loose<quad, sizeof(raw)>::type*>(p + c + V * k) = __builtin_bit_cast(quad, o);
        }
    } else if (!WIDE) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (c + k < D) p[c + k] = to_raw<DT>(x[k]);
    }
}

// Which of the eight elements of (row, columns 8 c ..) are kept: bit k of the result. Philox4x32, ten rounds (J. Salmon
// et al., "Parallel random numbers: as easy as 1, 2, 3", 2011): four multiplications of 32 to 64 bits in the round, for
// eight elements of 16 bits.
__device__ __forceinline__ unsigned kept8(const long* seed, unsigned c, unsigned row, unsigned drop) {
    const unsigned long key = seed[0], off = seed[1];
    unsigned c0 = c, c1 = row, c2 = (unsigned)off, c3 = (unsigned)(off >> 32), k0 = (unsigned)key, k1 = (unsigned)(key >> 32);
#pragma unroll
    for (int k = 0; k < 10; ++k) {
        const unsigned long a = (unsigned long)c0 * 0xD2511F53u, b = (unsigned long)c2 * 0xCD9E8D57u;
        c0 = (unsigned)(b >> 32) ^ c1 ^ k0;
        c1 = (unsigned)b;
        c2 = (unsigned)(a >> 32) ^ c3 ^ k1;
        c3 = (unsigned)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    const unsigned w[4] = {c0, c1, c2, c3};
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m |= ((w[k] & 0xffffu) >= drop ? 1u : 0u) << (2 * k);
        m |= ((w[k] >> 16) >= drop ? 1u : 0u) << (2 * k + 1);
    }
    return m;
}

// ---------------------------------------------------------------- host side
// f<TPR, accesses a thread>
template <class F> mimo_status with_row(int64_t D, F f) {
    const int64_t nv = (D + NV - 1) / NV;
    if (nv <= 8) return f.template operator()<8, 1>();
    if (nv <= 16) return f.template operator()<16, 1>();
    if (nv <= 32) return f.template operator()<32, 1>();
    if (nv <= 64) return f.template operator()<64, 1>();
    if (nv <= 128) return f.template operator()<128, 1>();
    if (nv <= 1024) return f.template operator()<0, 1>();
    return f.template operator()<0, 2>();
}
// threads of a block, and its rows
struct RowShape {
    int threads, rows;
};
inline RowShape shape_of(int64_t D) {
    const int nv = (int)((D + NV - 1) / NV);
    if (nv <= 128) return {256, nv <= 8 ? 32 : nv <= 16 ? 16 : nv <= 32 ? 8 : nv <= 64 ? 4 : 2};
    const int each = nv <= 1024 ? 1 : 2;
    return {(nv + 64 * each - 1) / (64 * each) * 64, 1};
}
// f<type of the data, type of the stream, wide accesses>
template <class F> mimo_status with_types(int dtype, int wide_stream, bool even, F f) {
    if (dtype == F32) return even ? f.template operator()<F32, F32, true>() : f.template operator()<F32, F32, false>();
    if (dtype == BF16) {
        if (wide_stream) return even ? f.template operator()<BF16, F32, true>() : f.template operator()<BF16, F32, false>();
        return even ? f.template operator()<BF16, BF16, true>() : f.template operator()<BF16, BF16, false>();
    }
    if (wide_stream) return even ? f.template operator()<F16, F32, true>() : f.template operator()<F16, F32, false>();
    return even ? f.template operator()<F16, F16, true>() : f.template operator()<F16, F16, false>();
}
inline mimo_status check_add_norm(int64_t rows, int64_t D, int dtype, float eps, int drop, const void* seed) {
    if (rows < 1 || D < 1) return bad("rows and channels must be positive");
    if (dtype < BF16 || dtype > F32) return set_error(MIMO_ERR_TYPE, "dtype must be a MIMO_DTYPE_* code");
    if (!(eps >= 0.f)) return bad("eps must not be negative");
    if (drop < 0 || drop > 65535) return bad("drop must be in [0, 65535]");
    if (drop && !seed) return bad("dropout needs a seed");
    if (D > MAMBA_ADD_NORM_MAX_WIDTH) return unsupported("more than 16384 channels");
    if (rows > (int64_t)1 << 31) return unsupported("more than 2^31 rows");
    return MIMO_OK;
}
inline float drop_factor(int drop) { return 65536.f / (float)(65536 - drop); }

}  // namespace layer
}  // namespace mimo
