// kda_linear_device.h -- device helpers of the linear-rule and tree kernels.
#pragma once
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_linear.h"

namespace kda {
namespace lin {

typedef double f64x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Token range of piece j of document n; pieces of `piece` tokens, piece = 0 for the whole
// document.  Every bound is clamped to [0, T], so a malformed cu cannot address memory
// outside the buffers.
struct Range {
    int64_t lo, hi, start, end;   // the piece and its document
    int n, j;
};
__device__ __forceinline__ void doc_bounds(const int32_t* cu, int seqlen, int64_t T, int n, int64_t& s, int64_t& e) {
    s = cu ? (int64_t)cu[n] : (int64_t)n * seqlen;
    e = cu ? (int64_t)cu[n + 1] : s + seqlen;
    s = s < 0 ? 0 : (s > T ? T : s);
    e = e < s ? s : (e > T ? T : e);
}
__device__ __forceinline__ int piece_owner(const int32_t* cu, int N, int seqlen, int64_t slot, int piece) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int64_t start = cu ? (int64_t)cu[mid] : (int64_t)mid * seqlen;
        if (start / piece + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ Range piece_range(const int32_t* cu, int N, int seqlen, int64_t T, int64_t slot, int piece) {
    Range r;
    if (piece == 0) {
        r.n = (int)slot;
        r.j = 0;
        doc_bounds(cu, seqlen, T, r.n, r.start, r.end);
        r.lo = r.start;
        r.hi = r.end;
        return r;
    }
    r.n = piece_owner(cu, N, seqlen, slot, piece);
    doc_bounds(cu, seqlen, T, r.n, r.start, r.end);
    r.j = (int)(slot - r.start / piece - r.n);
    if (r.j < 0) r.j = 0;
    r.lo = r.start + (int64_t)r.j * piece;
    r.hi = r.lo + piece;
    if (r.lo > r.end) r.lo = r.end;
    if (r.hi > r.end) r.hi = r.end;
    return r;
}

// A token's gate in log2 units.  Below -128 e^g is zero in fp32 either way (the smallest
// fp32 value is e^-103), so such gates, -inf among them, count as -128: every difference of
// sums stays finite.  NaN stays NaN.
__device__ __forceinline__ double gate_log2(float g) { return (double)(g < -128.f ? -128.f : g) * 1.4426950408889634; }

// Inclusive sum over the 64 lanes.  64 bits: the decay between two tokens is the difference
// of two sums, and sums of strong gates would leave fp32 differences only ~1e-4 exact.
__device__ __forceinline__ double wave_scan(double x, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(x, d, 64);
        if (lane >= d) x += y;
    }
    return x;
}

// Fragment of the transpose of a row-major tile: elements 0..3 are rows r0..r0+3 and 4..7
// rows r1..r1+3 of column c0 + lane % 16.  16-bit elements go through the LDS transpose
// read (each lane names four columns of one row; see lds_tr4 in kda_f16.h), 32-bit ones
// are read one by one.
__device__ __forceinline__ bf16x4 tr4(const bf16* p) {
    typedef short v4s __attribute__((__vector_size__(4 * sizeof(short))));
    const v4s r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(const_cast<bf16*>(p)));
    return __builtin_bit_cast(bf16x4, r);
}
__device__ __forceinline__ bf16x8 col_frag(const bf16* t, int ld, int r0, int r1, int c0, int cl) {
    const bf16* p = t + (cl >> 2) * ld + c0 + 4 * (cl & 3);
    const bf16x4 a = tr4(p + r0 * ld), b = tr4(p + r1 * ld);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x8 col_frag(const float* t, int ld, int r0, int r1, int c0, int cl) {
    f32x8 x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = t[(r0 + j) * ld + c0 + cl];
        x[j + 4] = t[(r1 + j) * ld + c0 + cl];
    }
    return x;
}
// Two groups of four contiguous elements: the k order of two stacked accumulator blocks.
template <typename T> __device__ __forceinline__ typename V8<T>::t two4(const T* a, const T* b) {
    const typename V4<T>::t x = lds4<T>(a), y = lds4<T>(b);
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x8 widen8(bf16x8 x) { return __builtin_convertvector(x, f32x8); }
__device__ __forceinline__ f32x8 widen8(f32x8 x) { return x; }

// c += a^T-operand x * b where x is an fp32 fragment.  bf16: x enters as three bf16 terms
// (24 bits), so that fp32 states and state gradients keep fp32 accuracy; fp32: exact.
template <bool X_IS_A> __device__ __forceinline__ f32x4 mma_f32x(f32x4 c, f32x8 x, bf16x8 b) {
    bf16x8 h = __builtin_convertvector(x, bf16x8);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        c = X_IS_A ? mma_k32(c, h, b) : mma_k32(c, b, h);
        if (i < 2) {
            x -= __builtin_convertvector(h, f32x8);
            h = __builtin_convertvector(x, bf16x8);
        }
    }
    return c;
}

template <bool X_IS_A> __device__ __forceinline__ f32x4 mma_f32x(f32x4 c, f32x8 x, f32x8 b) {
    return X_IS_A ? mma_k32(c, x, b) : mma_k32(c, b, x);
}

__device__ __forceinline__ void store4(void* base, int64_t at, f32x4 x, int out_bf16) {
    if (out_bf16) *reinterpret_cast<bf16x4*>((bf16*)base + at) = pack4<bf16>(x);
    else *reinterpret_cast<f32x4*>((float*)base + at) = x;
}
__device__ __forceinline__ void store1(void* base, int64_t at, float x, int out_bf16) {
    if (out_bf16) ((bf16*)base)[at] = (bf16)x;
    else ((float*)base)[at] = x;
}

// A tile of ROWS x COLS (row-major in global with row stride `ld` elements) held in
// registers between its loads and its LDS stores, 16 bytes a piece.  Rows at or past
// `rows` are read from the last valid row and stored as zeros.
template <typename T, int ROWS, int COLS, int THREADS> struct Tile {
    static constexpr int E = 16 / (int)sizeof(T);            // elements per piece
    static constexpr int PR = COLS / E;                       // pieces per row
    static constexpr int PIECES = ROWS * PR / THREADS;
    static_assert(ROWS * PR % THREADS == 0, "tile pieces");
    typedef unsigned u4 __attribute__((ext_vector_type(4)));
    u4 r[PIECES];
    __device__ __forceinline__ void load(const T* g, int64_t ld, int rows, int tid) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int x = tid + i * THREADS, row = x / PR, c = x % PR;
            const int rr = row < rows ? row : rows - 1;
            r[i] = *reinterpret_cast<const u4*>(g + (int64_t)rr * ld + c * E);
        }
    }
    __device__ __forceinline__ void store(T* s, int lds, int rows, int tid) const {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int x = tid + i * THREADS, row = x / PR, c = x % PR;
            const u4 z = {0u, 0u, 0u, 0u};
            *reinterpret_cast<u4*>(s + row * lds + c * E) = row < rows ? r[i] : z;
        }
    }
};

}  // namespace lin
}  // namespace kda
