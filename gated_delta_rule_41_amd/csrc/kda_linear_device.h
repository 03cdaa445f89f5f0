// kda_linear_device.h -- device helpers of the linear-rule and tree kernels.
#pragma once
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_linear.h"

namespace kda {
namespace lin {


// A lane value the compiler cannot see through: LDS offsets made from it stay inside the loop
// (a few integer operations) instead of being kept in registers across it.
__device__ __forceinline__ int opaque(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

// Token range of a piece of a document.  Every bound is clamped to [0, T], so a malformed cu cannot address memory
// outside the buffers.
struct Range {
    int64_t lo, hi, start, end;   // the piece and its document
    int n;
};
__device__ __forceinline__ void doc_bounds(const int32_t* cu, int seqlen, int64_t T, int n, int64_t& s, int64_t& e) {
    s = cu ? (int64_t)cu[n] : (int64_t)n * seqlen;
    e = cu ? (int64_t)cu[n + 1] : s + seqlen;
    s = s < 0 ? 0 : (s > T ? T : s);
    e = e < s ? s : (e > T ? T : e);
}
// The document that owns `slot` when document n's pieces start at slot start / piece + n:
// the last n whose first slot is not past it.  Every lane of the wave takes part: 64
// documents are looked at per load, where a binary search would wait for one load per halving.
__device__ __forceinline__ int piece_owner(const int32_t* cu, int N, int seqlen, int64_t slot, int piece) {
    const int l = threadIdx.x & 63;
    int lo = 0, n = N;
    while (true) {
        const int step = (n + 63) / 64, i = lo + l * step;
        bool past = true;
        if (l * step < n) {
            const int64_t start = cu ? (int64_t)cu[i] : (int64_t)i * seqlen;
            past = start / piece + i > slot;
        }
        const unsigned long long m = __ballot(!past);
        const int last = m ? 63 - __clzll((long long)m) : 0;
        lo += last * step;
        n = n - last * step < step ? n - last * step : step;
        if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
    }
}
__device__ __forceinline__ Range piece_range(const int32_t* cu, int N, int seqlen, int64_t T, int64_t slot, int piece) {
    Range r;
    r.n = piece_owner(cu, N, seqlen, slot, piece);
    doc_bounds(cu, seqlen, T, r.n, r.start, r.end);
    int64_t j = slot - r.start / piece - r.n;
    if (j < 0) j = 0;
    r.lo = r.start + j * piece;
    r.hi = r.lo + piece;
    if (r.lo > r.end) r.lo = r.end;
    if (r.hi > r.end) r.hi = r.end;
    return r;
}

// Segments of seg_len tokens are numbered through the documents without gaps (an empty
// document has one), so that the workgroups of a walk that have nothing to do are the last
// ones: spread among the others they would leave some compute units with all of the work.
// Every lane takes part, 64 documents at a time (at most kSegDocs of them).
__device__ __forceinline__ int wave_scan_int(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}
__device__ __forceinline__ int doc_segments(const int32_t* cu, int seqlen, int64_t T, int n, int seg_len) {
    int64_t s, e;
    doc_bounds(cu, seqlen, T, n, s, e);
    const int c = (int)((e - s + seg_len - 1) / seg_len);
    return c > 1 ? c : 1;
}
// The number of segments before document n.
__device__ __forceinline__ int segments_before(const int32_t* cu, int seqlen, int64_t T, int seg_len, int n) {
    const int l = threadIdx.x & 63;
    int before = 0;
    for (int n0 = 0; n0 < n; n0 += 64)
        before += __builtin_amdgcn_readlane(wave_scan_int(n0 + l < n ? doc_segments(cu, seqlen, T, n0 + l, seg_len) : 0), 63);
    return before;
}
// Segment k, or document k as a whole with seg_len = 0; r.n = N where there is none.
__device__ __forceinline__ Range seg_range(const int32_t* cu, int N, int seqlen, int64_t T, int64_t k, int seg_len) {
    Range r;
    int64_t j = 0;
    r.n = (int)k;
    if (seg_len) {
        const int l = threadIdx.x & 63;
        int64_t left = k;
        r.n = N;
        for (int n0 = 0; n0 < N; n0 += 64) {
            const int c = n0 + l < N ? doc_segments(cu, seqlen, T, n0 + l, seg_len) : 0;
            const int upto = wave_scan_int(c), all = __builtin_amdgcn_readlane(upto, 63);
            if (left < all) {
                const int at = __ffsll((long long)__ballot(upto > left)) - 1;
                r.n = n0 + at;
                j = left - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(c, at));
                break;
            }
            left -= all;
        }
        if (r.n == N) {
            r.lo = r.hi = r.start = r.end = 0;
            return r;
        }
    }
    doc_bounds(cu, seqlen, T, r.n, r.start, r.end);
    r.lo = seg_len ? r.start + j * seg_len : r.start;
    r.hi = seg_len && r.lo + seg_len < r.end ? r.lo + seg_len : r.end;
    return r;
}

// Documents of up to whole_len tokens each stay whole; if one is longer, all are cut into seg_len.
// (A launch's walks end together with documents alike, and cutting them would only cost; with
// documents unlike, the shorter segments even them out.)
__device__ __forceinline__ int segment_length(const int32_t* cu, int N, int seqlen, int64_t T, int seg_len, int whole_len) {
    const int l = threadIdx.x & 63;
    if (!whole_len) return seg_len;
    for (int n0 = 0; n0 < N; n0 += 64) {
        int64_t s = 0, e = 0;
        if (n0 + l < N) doc_bounds(cu, seqlen, T, n0 + l, s, e);
        if (__ballot(e - s > whole_len)) return seg_len;
    }
    return whole_len;
}

// The k-th longest segment of up to 64 documents: all full ones in the documents' order, then
// their rests from the longest on (an empty document's is empty), so that a launch of unlike
// walks ends evenly.  `slot` is the segment's number as in seg_range.  A rest's key holds its
// length in 1024ths of a segment and its document, and the wanted one is found bit by bit: the
// largest key that more than k - (full segments) rests reach.
__device__ __forceinline__ Range longest_range(const int32_t* cu, int N, int seqlen, int64_t T, int64_t k, int seg_len, int64_t& slot) {
    const int l = threadIdx.x & 63;
    Range r;
    int full = 0, key = 0, segments = 0;
    if (l < N) {
        int64_t s, e;
        doc_bounds(cu, seqlen, T, l, s, e);
        full = (int)((e - s) / seg_len);
        const int64_t rest = (e - s) - (int64_t)full * seg_len;
        const bool any = rest || s == e;
        if (any) key = (int)(rest * 1024 / seg_len << 6 | (63 - l)) + 1;
        segments = full + any;
    }
    const int upto = wave_scan_int(full), all = __builtin_amdgcn_readlane(upto, 63);
    int64_t j;
    if (k < all) {
        r.n = __ffsll((long long)__ballot(upto > k)) - 1;
        j = k - (__builtin_amdgcn_readlane(upto, r.n) - __builtin_amdgcn_readlane(full, r.n));
    } else {
        int found = 0;
        for (int bit = 1 << 16; bit; bit >>= 1)
            if (__popcll(__ballot(key >= (found | bit))) > k - all) found |= bit;
        if (!found) {
            r.lo = r.hi = r.start = r.end = 0;
            r.n = N;
            return r;
        }
        r.n = 63 - ((found - 1) & 63);
        j = __builtin_amdgcn_readlane(full, r.n);
    }
    doc_bounds(cu, seqlen, T, r.n, r.start, r.end);
    r.lo = r.start + j * seg_len;
    r.hi = r.lo + seg_len < r.end ? r.lo + seg_len : r.end;
    slot = __builtin_amdgcn_readlane(wave_scan_int(segments) - segments, r.n) + j;
    return r;
}

// A token's gate in log2 units.  Below -128 e^g is zero in fp32 either way (the smallest
// fp32 value is e^-103), so such gates, -inf among them, count as -128: every difference of
// sums stays finite.  NaN stays NaN.
__device__ __forceinline__ double gate_log2(float g) { return (double)(g < -128.f ? -128.f : g) * 1.4426950408889634; }

// Inclusive sum over the 64 lanes, by data-parallel moves within and across rows of 16 (no
// LDS round trips: the scan sits on a chunk's critical path).  64 bits: the decay between two
// tokens is the difference of two sums, and sums of strong gates would leave fp32
// differences only ~1e-4 exact.  Every lane must be active.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp64(double x) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    const i32x2 v = __builtin_bit_cast(i32x2, x);
    i32x2 r;
    r[0] = __builtin_amdgcn_update_dpp(0, v[0], CTRL, ROWS, 0xF, false);
    r[1] = __builtin_amdgcn_update_dpp(0, v[1], CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, r);
}
__device__ __forceinline__ double wave_scan(double x) {
    x += dpp64<0x111, 0xF>(x);   // row_shr 1, 2, 4, 8: sums within each row of 16
    x += dpp64<0x112, 0xF>(x);
    x += dpp64<0x114, 0xF>(x);
    x += dpp64<0x118, 0xF>(x);
    x += dpp64<0x142, 0xA>(x);   // row_bcast 15 into rows 1 and 3
    x += dpp64<0x143, 0xC>(x);   // row_bcast 31 into rows 2 and 3
    return x;
}
__device__ __forceinline__ double last_lane(double x) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    i32x2 v = __builtin_bit_cast(i32x2, x);
    v[0] = __builtin_amdgcn_readlane(v[0], 63);
    v[1] = __builtin_amdgcn_readlane(v[1], 63);
    return __builtin_bit_cast(double, v);
}

// Row-major LDS tile without padding, its 16-byte pieces permuted inside each row by
// piece ^ swz(row).  LDS reads see 64 banks, 16 lanes a cycle for 16-byte reads and 32 for
// 8-byte and transpose reads.  With r3..r0 the low bits of the row, the permutations below
// are one to one over 16 rows, so 16-byte reads of one piece of 16 rows touch every bank
// once, and they move eight rows r..r+3, r+4..r+7 (or r+8..r+11) to eight different pairs of
// pieces, so transpose reads of 16 columns do too.  (With rows padded by 16 bytes instead the
// transpose reads were 2-way conflicts.)
template <typename T, int COLS> struct Swz {
    static constexpr int E = 16 / (int)sizeof(T), PR = COLS / E;   // elements per piece, pieces per row
    static __device__ __forceinline__ int swz(int r) {
        if constexpr (sizeof(T) == 4) return r & 15;
        else if constexpr (PR == 16) return (r & 3) << 2 | (((r >> 2) ^ (r >> 3)) & 1) << 1 | ((r >> 3) & 1);
        else return ((r >> 1) & 1) << 2 | (((r >> 2) ^ (r >> 3)) & 1) << 1 | ((r >> 3) & 1);
    }
    static __device__ __forceinline__ int at(int row, int piece) { return row * COLS + (piece ^ swz(row)) * E; }
};

__device__ __forceinline__ bf16x4 tr4(const bf16* p) {
    typedef short v4s __attribute__((__vector_size__(4 * sizeof(short))));
    const v4s r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(const_cast<bf16*>(p)));
    return __builtin_bit_cast(bf16x4, r);
}
template <typename V> __device__ __forceinline__ auto join(V a, V b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// A lane's byte offsets into a Swz tile, and the product fragments read through them.  With
// `off` the byte offset of the first row (a multiple of 16 rows):
//   row(y):  columns 32 y + 8 qg + j of row cl
//   perm(y): columns 32 y + 4 qg + j and 32 y + 16 + 4 qg + j of row cl, the k order of two
//            stacked accumulator blocks
//   col(m):  rows 4 qg + j and 16 + 4 qg + j of column 16 m + cl, the same order by rows
// The permutation makes every further fragment of a row an exclusive-or of one lane constant
// with a literal.  16-bit columns go through the LDS transpose read (each lane names four
// columns of one row; see lds_tr4 in kda_f16.h), 32-bit ones are read one by one.
template <typename V> __device__ __forceinline__ V at_byte(const void* t, int off) {
    return *reinterpret_cast<const V*>((const char*)t + off);
}
template <typename T, int COLS> struct Lane;
template <int COLS> struct Lane<bf16, COLS> {
    typedef Swz<bf16, COLS> Z;
    static constexpr int RB = COLS * 2;   // bytes per row
    int r, p, c;
    __device__ __forceinline__ Lane(int cl, int qg) {
        const int cr = 4 * qg + (cl >> 2);
        r = cl * RB + (qg ^ Z::swz(cl)) * 16;
        p = cl * RB + ((qg >> 1) ^ Z::swz(cl)) * 16 + 8 * (qg & 1);
        c = cr * RB + (((cl >> 1) & 1) ^ Z::swz(cr)) * 16 + 8 * (cl & 1);
    }
    __device__ __forceinline__ bf16x8 row(const bf16* t, int off, int y) const { return at_byte<bf16x8>(t, (r + off) ^ (64 * y)); }
    __device__ __forceinline__ bf16x8 perm(const bf16* t, int off, int y) const {
        return join(at_byte<bf16x4>(t, (p + off) ^ (64 * y)), at_byte<bf16x4>(t, (p + off) ^ (64 * y + 32)));
    }
    __device__ __forceinline__ bf16x8 col(const bf16* t, int off, int m) const {
        const bf16* x = (const bf16*)((const char*)t + ((c + off) ^ (32 * m)));
        return join(tr4(x), tr4(x + 16 * COLS));
    }
};
template <int COLS> struct Lane<float, COLS> {
    typedef Swz<float, COLS> Z;
    static constexpr int RB = COLS * 4;
    int r, p, c[4];
    __device__ __forceinline__ Lane(int cl, int qg) {
        r = cl * RB + ((2 * qg) ^ Z::swz(cl)) * 16;
        p = cl * RB + (qg ^ Z::swz(cl)) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = (4 * qg + j) * RB + ((cl >> 2) ^ Z::swz(4 * qg + j)) * 16 + 4 * (cl & 3);
    }
    __device__ __forceinline__ f32x8 row(const float* t, int off, int y) const {
        return join(at_byte<f32x4>(t, (r + off) ^ (128 * y)), at_byte<f32x4>(t, (r + off) ^ (128 * y + 16)));
    }
    __device__ __forceinline__ f32x8 perm(const float* t, int off, int y) const {
        return join(at_byte<f32x4>(t, (p + off) ^ (128 * y)), at_byte<f32x4>(t, (p + off) ^ (128 * y + 64)));
    }
    __device__ __forceinline__ f32x8 col(const float* t, int off, int m) const {
        f32x8 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = (c[j] + off) ^ (64 * m);
            x[j] = at_byte<float>(t, o);
            x[j + 4] = at_byte<float>(t, o + 16 * RB);
        }
        return x;
    }
};
// Where four accumulator values (row cl, columns 16 n + 4 qg + i) go in a tile.
template <typename T, int COLS> __device__ __forceinline__ void put4(T* t, int row, int n, int qg, f32x4 x) {
    typedef Swz<T, COLS> Z;
    if constexpr (sizeof(T) == 2) sts4(t + Z::at(row, 2 * n + (qg >> 1)) + 4 * (qg & 1), x);
    else sts4(t + Z::at(row, 4 * n + qg), x);
}
// x where `on`, else 0, without a branch (a branch around the few instructions that make x
// costs more than they do).
__device__ __forceinline__ float keep(float x, bool on) {
    return __builtin_bit_cast(float, __builtin_bit_cast(int, x) & (on ? -1 : 0));
}

// From the bits (unpack4), so that the compiler does not rebuild values by conversions.
__device__ __forceinline__ f32x8 widen8(bf16x8 x) {
    return join(unpack4(__builtin_shufflevector(x, x, 0, 1, 2, 3)), unpack4(__builtin_shufflevector(x, x, 4, 5, 6, 7)));
}
__device__ __forceinline__ f32x8 widen8(f32x8 x) { return x; }

// Infinities and NaN.  A result that depends on one is never finite again, but the zeros of a
// causal mask times one would be NaN too.  So where a tile holds any, products behind a mask take
// the finite values alone, and the results that the others reach become NaN.

// t, which is 0, or NaN where one of 16 bytes' values is infinite or NaN: zero times it is not zero.
template <typename T> __device__ __forceinline__ float probe(u32x4 x, float t) {
    if constexpr (sizeof(T) == 2) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, (unsigned)x[i]), bf16x2{0, 0}, t, false);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) t = __builtin_fmaf(__uint_as_float(x[i]), 0.f, t);
    }
    return t;
}
// All ones where a value is infinite or NaN.
__device__ __forceinline__ u16x8 not_finite(bf16x8 x) { return (u16x8)((__builtin_bit_cast(u16x8, x) & (unsigned short)0x7f80) == (unsigned short)0x7f80); }
__device__ __forceinline__ u32x8 not_finite(f32x8 x) { return (u32x8)((__builtin_bit_cast(u32x8, x) & 0x7f800000u) == 0x7f800000u); }
// The finite values, zeros in the place of the others.
template <typename V> __device__ __forceinline__ V finite_part(V x) {
    const auto m = not_finite(x);
    return __builtin_bit_cast(V, __builtin_bit_cast(decltype(not_finite(x)), x) & ~m);
}
template <typename T> __device__ __forceinline__ u32x4 finite_piece(u32x4 x) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(u32x4, finite_part(__builtin_bit_cast(bf16x8, x)));
    else return x & ~(u32x4)((x & 0x7f800000u) == 0x7f800000u);
}
// For a transposed tile's fragment x (32 rows in the k order of Lane::col): in the accumulator
// layout, how many values of each of its columns are infinite or NaN among the rows that reach(row).
template <typename V, typename F> __device__ __forceinline__ f32x4 odd_count(V x, int qg, F&& reach) {
    const auto m = not_finite(x);
    V odd, mask;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        odd[e] = m[e] ? 1.f : 0.f;
        mask[e] = reach((e < 4 ? 0 : 12) + 4 * qg + e) ? 1.f : 0.f;
    }
    return mma_k32(zero4(), odd, mask);
}

// c + x y for a transposed tile's fragment x and weights y that are zero in the columns that a row
// does not reach: x's infinities and NaN make NaN of what their row reaches, and nothing of the rest.
template <typename V, typename F> __device__ __forceinline__ f32x4 mma_reaching(f32x4 c, V x, V y, int qg, F&& reach) {
    c = mma_k32(c, finite_part(x), y);
    const f32x4 odd = odd_count(x, qg, reach);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = odd[i] > 0.f ? __builtin_nanf("") : c[i];
    return c;
}

// An fp32 fragment as a product operand.  bf16: three bf16 terms (24 bits), so that fp32
// states and state gradients keep fp32 accuracy; fp32: itself.  (The terms of an infinity are
// one and NaN.)
template <typename T> struct Split;
template <> struct Split<bf16> {
    bf16x8 h[3];
    __device__ __forceinline__ Split() {}
    __device__ __forceinline__ explicit Split(f32x8 x) {
        h[0] = __builtin_convertvector(x, bf16x8);
        x -= widen8(h[0]);
        h[1] = __builtin_convertvector(x, bf16x8);
        x -= widen8(h[1]);
        h[2] = __builtin_convertvector(x, bf16x8);
    }
    static constexpr int TERMS = 3;
    template <bool IS_A> __device__ __forceinline__ f32x4 mma(int i, f32x4 c, bf16x8 b) const {   // term i, smallest first
        return IS_A ? mma_k32(c, h[2 - i], b) : mma_k32(c, b, h[2 - i]);
    }
};
template <> struct Split<float> {
    f32x8 x;
    __device__ __forceinline__ Split() {}
    __device__ __forceinline__ explicit Split(f32x8 y) : x(y) {}
    static constexpr int TERMS = 1;
    template <bool IS_A> __device__ __forceinline__ f32x4 mma(int, f32x4 c, f32x8 b) const {
        return IS_A ? mma_k32(c, x, b) : mma_k32(c, b, x);
    }
};

__device__ __forceinline__ void store4(void* base, int64_t at, f32x4 x, int out_bf16) {
    if (out_bf16) *reinterpret_cast<bf16x4*>((bf16*)base + at) = pack4<bf16>(x);
    else *reinterpret_cast<f32x4*>((float*)base + at) = x;
}
__device__ __forceinline__ void store1(void* base, int64_t at, float x, int out_bf16) {
    if (out_bf16) ((bf16*)base)[at] = (bf16)x;
    else ((float*)base)[at] = x;
}

// `rows` rows of `cols` elements with stride `ld`, as a buffer: reads past its end return zeros
// and writes past it are dropped, so rows behind a document's end need no branches.  That
// matters beyond the branches: a wait for one load must count the memory operations issued
// after it, and around conditional ones the compiler can only wait for all of them.
// At most 128 rows (checked on the host to be below 2^31 bytes); `base` and the counts are
// the same for the whole wave.
typedef __amdgpu_buffer_rsrc_t Buffer;
template <typename T> __device__ __forceinline__ Buffer rows_of(const T* base, int64_t ld, int rows, int most, int cols) {
    const int n = rows < 0 ? 0 : rows < most ? rows : most;
    const int bytes = n ? (int)((unsigned)((n - 1) * (int)ld + cols) * sizeof(T)) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, unsigned off) { return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0); }
template <typename T> __device__ __forceinline__ T load_one(Buffer b, unsigned at) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(bf16, (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(b, at * 2, 0, 0));
    else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, at * 4, 0, 0));
}
// Four values at element `at` of a buffer of O.
template <typename O> __device__ __forceinline__ void store4(Buffer b, unsigned at, f32x4 x) {
    if constexpr (sizeof(O) == 2) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, pack4<bf16>(x)), b, at * 2, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b, at * 4, 0, 0);
}
// Rows 0 and 1 of 16 lanes, and 2 and 3, trade: what lane qg of a has of the first 16 columns
// (4 qg ..) and of b of the second becomes 8 columns in a row, from trade_col(qg) on; and back.
__device__ __forceinline__ u32x4 trade(u32x2 a, u32x2 b) {
    const auto lo = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false), hi = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    return u32x4{lo[0], hi[0], lo[1], hi[1]};
}
__device__ __forceinline__ int trade_col(int qg) { return 16 * (qg & 1) + 8 * (qg >> 1); }
__device__ __forceinline__ u32x4 trade_bf16(f32x4 x, f32x4 y) {
    return trade(__builtin_bit_cast(u32x2, pack4<bf16>(x)), __builtin_bit_cast(u32x2, pack4<bf16>(y)));
}
// Two accumulator blocks side by side (x: four values at column 4 qg of a row's first 16, y: of
// its second) to 32 columns of a row from `at`.  bf16: each lane stores 16 bytes and a row 64 in
// a piece, where 8 and 32 of them would be (memory takes pieces of rows worse the smaller they
// are: gradients of 4 x 8192 x 32 heads 753 -> 664 us).
template <typename O> __device__ __forceinline__ void store8(Buffer b, unsigned at, int qg, f32x4 x, f32x4 y) {
    if constexpr (sizeof(O) == 2) {
        __builtin_amdgcn_raw_buffer_store_b128(trade_bf16(x, y), b, (at + trade_col(qg)) * 2, 0, 0);
    } else {
        store4<O>(b, at + 4 * qg, x);
        store4<O>(b, at + 16 + 4 * qg, y);
    }
}
// Row `row` of D columns, four values at 16 m + 4 qg for every m, to a block's output of either
// type: one branch.
template <typename O, int D> __device__ __forceinline__ void store_row(O* base, int64_t ld, int rows, int most, int row, int qg, const f32x4 (&x)[D / 16]) {
    const Buffer b = rows_of(base, ld, rows, most, D);
#pragma unroll
    for (int m = 0; m < D / 16; m += 2) store8<O>(b, row * (unsigned)ld + 16 * m, qg, x[m], x[m + 1]);
}
template <int D> __device__ __forceinline__ void store_row(void* base, int64_t at, int64_t ld, int rows, int most, int row, int qg, const f32x4 (&x)[D / 16], int out_bf16) {
    if (out_bf16) store_row<bf16, D>((bf16*)base + at, ld, rows, most, row, qg, x);
    else store_row<float, D>((float*)base + at, ld, rows, most, row, qg, x);
}

// A tile of ROWS x COLS (row-major in global with row stride `ld` elements) held in registers
// between its loads and its stores to a Swz tile, 16 bytes a piece.  Rows at or past `rows`
// are zeros.
template <typename T, int ROWS, int COLS, int THREADS> struct Tile {
    typedef Swz<T, COLS> Z;
    static constexpr int PIECES = ROWS * Z::PR / THREADS, STEP = THREADS / Z::PR;   // rows between a lane's pieces
    static_assert(ROWS * Z::PR % THREADS == 0, "tile pieces");
    u32x4 r[PIECES];
    __device__ __forceinline__ void load(const T* g, int64_t ld, int rows, int tid) {
        const Buffer b = rows_of(g, ld, rows, ROWS, COLS);
        const unsigned row = (unsigned)ld * sizeof(T), off = (unsigned)(tid / Z::PR) * row + (tid % Z::PR) * 16u;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) r[i] = load16(b, off + i * STEP * row);
    }
    __device__ __forceinline__ void store(T* s, int tid) const {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) *reinterpret_cast<u32x4*>(s + Z::at(tid / Z::PR + i * STEP, tid % Z::PR)) = r[i];
    }
};

}  // namespace lin
}  // namespace kda
