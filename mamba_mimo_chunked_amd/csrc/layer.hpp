// What the layer operators (layer_*.hip) share: element types, the placement of
// sequences and chunks, fp32 functions, lane exchanges, sums over partial rows and
// the host's launch and error helpers.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "mamba_layer.h"

namespace mimo {

// host side, defined in mimo_bwd_fwd.hip: the thread's error message, the device check
mimo_status set_error(mimo_status s, const char* msg);
mimo_status require_gfx950();

namespace layer {

constexpr int BF16 = MIMO_DTYPE_BF16, F16 = MIMO_DTYPE_FP16, F32 = MIMO_DTYPE_FP32;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// ---------------------------------------------------------------- elements
template <int DT> struct Elem { typedef unsigned short raw; };
template <> struct Elem<F32> { typedef float raw; };
template <int DT> using raw_t = typename Elem<DT>::raw;
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));

template <int DT> __device__ __forceinline__ float to_f(raw_t<DT> r) {
    if constexpr (DT == F32) return r;
    else if constexpr (DT == BF16) return __uint_as_float((unsigned)r << 16);
    else return (float)__builtin_bit_cast(_Float16, r);
}
template <int DT> __device__ __forceinline__ raw_t<DT> to_raw(float x) {
    if constexpr (DT == F32) return x;
    else if constexpr (DT == BF16) return (unsigned short)__builtin_bit_cast(unsigned, __builtin_convertvector(f2{x, 0.f}, b16x2));
    else return __builtin_bit_cast(unsigned short, (_Float16)x);
}
// VEC consecutive elements, loaded or stored as one access of up to 16 bytes
template <int DT, int VEC> struct alignas(sizeof(raw_t<DT>) * VEC) Pack { raw_t<DT> v[VEC]; };
template <int DT, int VEC> __device__ __forceinline__ Pack<DT, VEC> load(const raw_t<DT>* p) {
    return *reinterpret_cast<const Pack<DT, VEC>*>(p);
}
template <int DT, int VEC> __device__ __forceinline__ void store(raw_t<DT>* p, const float (&x)[VEC]) {
    Pack<DT, VEC> o;
#pragma unroll
    for (int i = 0; i < VEC; ++i) o.v[i] = to_raw<DT>(x[i]);
    *reinterpret_cast<Pack<DT, VEC>*>(p) = o;
}
template <int DT, int VEC> __device__ __forceinline__ void unpack(const Pack<DT, VEC>& r, float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = to_f<DT>(r.v[i]);
}

// ---------------------------------------------------------------- fp32 functions
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp2_hw(-LOG2E * x)); }
// d silu(x) / dx from g = sigmoid(x)
__device__ __forceinline__ float silu_slope(float x, float g) { return g * __builtin_fmaf(x, 1.f - g, 1.f); }
// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|). The rounding of |x| log2(e) is put back into e, and that of
// w = 1 + e behind the logarithm: log1p(e) = log(w) + (e - (w - 1)) / w, with w = 1 where the second term counts. So
// small step sizes keep their relative precision (2.6e-7 at most, 5e-8 root mean square on [-20, 20]; hardware exp2
// and log2). Beyond |x| = 100, e is below fp32's range. NaN passes through the first term.
__device__ __forceinline__ float softplus(float x) {
    const float m = __builtin_fminf(__builtin_fabsf(x), 100.f), hi = -LOG2E * m;
    float e = exp2_hw(hi);
    e = __builtin_fmaf(e, __builtin_fmaf(hi, -LN2, -m), e);
    const float w = 1.f + e;
    return (x < 0.f ? 0.f : x) + __builtin_fmaf(__builtin_amdgcn_logf(w), LN2, e - (w - 1.f));
}

// ---------------------------------------------------------------- lane exchanges
// Adds a value of another lane of the same 16-lane row: xor 1, 2 (quad permutations), xor 8
// (rotation by 8), and rotation by 4 (xor 4 for values that repeat every 8 lanes).
template <int CTRL> __device__ __forceinline__ float add_dpp(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_ROR4 = 0x124, DPP_ROR8 = 0x128, DPP_HALF_MIRROR = 0x141;
// xor 4: the half row mirrored, then each quad
__device__ __forceinline__ float add_xor4(float x) {
    const int m = __builtin_amdgcn_update_dpp(0, __float_as_int(x), DPP_HALF_MIRROR, 0xf, 0xf, true);
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, m, 0x1B, 0xf, 0xf, true));
}
typedef unsigned u2 __attribute__((ext_vector_type(2)));
// a and b of all lanes -> lanes 0-31: a + a of lane + 32; lanes 32-63: b + b of lane - 32
__device__ __forceinline__ float fold32(float a, float b) {
    const u2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}
// the same over neighbouring 16-lane rows: even rows sum a, odd rows sum b
__device__ __forceinline__ float fold16(float a, float b) {
    const u2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}
// and over 8-lane halves of a row: lanes with bit 3 clear sum a, set sum b
__device__ __forceinline__ float fold8(float a, float b, bool bit3) {
    const float keep = bit3 ? b : a, give = bit3 ? a : b;
    return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), DPP_ROR8, 0xf, 0xf, true));
}
// the sum over the Q lanes that share a channel (lane % Q), Q a power of two up to 16, in all of them
template <int Q> __device__ __forceinline__ float sum_lanes(float x) {
    if constexpr (Q >= 2) x = add_dpp<DPP_XOR1>(x);
    if constexpr (Q >= 4) x = add_dpp<DPP_XOR2>(x);
    if constexpr (Q >= 8) x = add_dpp<DPP_HALF_MIRROR>(x);
    if constexpr (Q >= 16) x = add_dpp<DPP_ROR8>(x);
    return x;
}
// the sum over W = 8, 16, 32 or 64 neighbouring lanes, in all of them
template <int W> __device__ __forceinline__ float sum_wave(float x) {
    x = sum_lanes<W < 16 ? W : 16>(x);
    if constexpr (W >= 32) x += __shfl_xor(x, 16);
    if constexpr (W >= 64) x += __shfl_xor(x, 32);
    return x;
}

// ---------------------------------------------------------------- sequences and chunks
// n sequences in chunks of CH tokens. Dense: chunk j of sequence i is slot i * nc + j. Packed: the
// chunks of sequence i take the slots from start(i) / CH + i on, which leaves each at least one and
// never more than it needs by one; the tokens behind the last sequence count as sequence n.
struct Seqs {
    const int* cu;
    int n, S, CH, nc;
    __device__ __forceinline__ int start(int i) const { return i == 0 ? 0 : min(max(cu[i], 0), S); }
    __device__ __forceinline__ int base(int i) const { return start(i) / CH + i; }
};
struct Place {
    int i, j;       // sequence (n: behind the last), chunk in it
    int row0, len;  // first token on the packed axis (0 when dense), length
    bool ok;        // the slot holds a chunk (the first one also where the sequence is empty)
};
__device__ __forceinline__ Place place(const Seqs& q, int slot) {
    Place r;
    if (q.cu == nullptr) {
        r.i = slot / q.nc;
        r.j = slot - r.i * q.nc;
        r.row0 = 0;
        r.len = q.S;
    } else {
        int lo = 0, hi = q.n;   // base(lo) <= slot throughout
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (q.base(mid) <= slot) lo = mid;
            else hi = mid - 1;
        }
        r.i = lo;
        r.j = slot - q.base(lo);
        r.row0 = q.start(lo);
        r.len = max((lo < q.n ? q.start(lo + 1) : q.S) - r.row0, 0);
    }
    r.ok = r.j == 0 || (long)r.j * q.CH < r.len;
    return r;
}
inline long slots_of(const Seqs& q) { return q.cu ? (long)q.S / q.CH + q.n + 1 : (long)q.n * q.nc; }

// a tensor with a batch and a token axis; packed: bs = 0
struct Rows {
    const void* p;
    long bs, ts;
};
template <int DT> __device__ __forceinline__ const raw_t<DT>* at(const Rows& r, const Place& pl) {
    return static_cast<const raw_t<DT>*>(r.p) + pl.i * r.bs + pl.row0 * r.ts;
}

// ---------------------------------------------------------------- rows that share a slot (steps)
// Whether `row` is the first with its index; if so it also takes the later rows of that index.
__device__ __forceinline__ bool first_of(const int* idx, int row, int slot) {
    const int lane = threadIdx.x & 63;
    for (int r0 = 0; r0 < row; r0 += 64) {
        const int r = r0 + lane;
        if (__ballot(r < row && idx[min(r, row)] == slot)) return false;
    }
    return true;
}
__device__ __forceinline__ int next_of(const int* idx, int row, int n, int slot) {
    const int lane = threadIdx.x & 63;
    for (int r0 = row + 1; r0 < n; r0 += 64) {
        const int r = r0 + lane;
        const unsigned long long m = __ballot(r < n && idx[min(r, n - 1)] == slot);
        if (m) return r0 + __builtin_ctzll(m);
    }
    return n;
}

// ---------------------------------------------------------------- sums over partial rows
// put(col, sum over R rows of part[r * ld + col]) for SUM_COLS columns from col0, by a block of 256 threads: sixteen
// threads a column, each over every sixteenth row with four sums in flight, joined in LDS in order.
// Few columns a block, so that the usual few thousand columns make enough blocks to fill the GPU.
constexpr int SUM_COLS = 16;
template <class F> __device__ __forceinline__ void column_sums(const float* part, long ld, long R, long col0, long cols, F put) {
    constexpr int TR = 256 / SUM_COLS;
    __shared__ float s[TR][SUM_COLS];
    const int c = threadIdx.x % SUM_COLS, w = threadIdx.x / SUM_COLS;
    const long col = col0 + c;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (col < cols) {
        const float* p = part + col;
        long r = w;
        for (; r + 3 * TR < R; r += 4 * TR) {
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] += p[(r + k * TR) * ld];
        }
        for (int k = 0; r < R; r += TR, ++k) acc[k] += p[r * ld];
    }
    s[w][c] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
    __syncthreads();
    if (w == 0 && col < cols) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < TR; ++k) x += s[k][c];
        put(col, x);
    }
}

// ---------------------------------------------------------------- host side
inline mimo_status bad(const char* msg) { return set_error(MIMO_ERR_VALUE, msg); }
inline mimo_status unsupported(const char* msg) { return set_error(MIMO_ERR_UNSUPPORTED, msg); }

// the most threads along a grid's first axis. A call of several kernels checks them all before it queues the first.
inline bool grid_fits(long blocks, int block) { return (unsigned long)blocks * block <= 0xffffffffUL; }
template <class P> inline mimo_status launch(void (*f)(P), dim3 grid, int block, size_t lds, hipStream_t st, P p) {
    if (!grid_fits(grid.x, block)) return unsupported("the call needs more than 2^32 threads");
    if (lds > 64 * 1024 && hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)lds) != hipSuccess)
        return set_error(MIMO_ERR_HIP, "hipFuncSetAttribute(MaxDynamicSharedMemorySize) failed");
    void* args[] = {&p};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(f), grid, dim3(block), args, lds, st);
    if (e != hipSuccess) return set_error(MIMO_ERR_HIP, hipGetErrorString(e));
    return MIMO_OK;
}

inline bool aligned(const void* p, int64_t s0, int64_t s1, int bytes, int esz) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s0 * esz % bytes == 0 && s1 * esz % bytes == 0;
}
inline Rows rows_of(const mamba_rows& r, bool packed) { return Rows{r.data, packed ? 0 : (long)r.batch_stride, (long)r.token_stride}; }
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

inline mimo_status check_sequences(int64_t n, int64_t S, int64_t D, int dtype) {
    if (n < 1 || S < 1 || D < 1) return bad("the numbers of sequences, tokens and channels must be positive");
    if (dtype < BF16 || dtype > F32) return set_error(MIMO_ERR_TYPE, "dtype must be a MIMO_DTYPE_* code");
    if (n > 65535) return unsupported("more than 65535 sequences");
    if (S > (int64_t)1 << 30) return unsupported("more than 2^30 tokens");
    if (D > (int64_t)1 << 20) return unsupported("more than 2^20 channels");
    return MIMO_OK;
}
inline mimo_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return MIMO_OK;
    if (ws == nullptr || have < need) return bad("workspace too small");
    if (reinterpret_cast<uintptr_t>(ws) % 256) return bad("workspace must be 256-byte aligned");
    return MIMO_OK;
}

}  // namespace layer
}  // namespace mimo
