// kda_layer.h -- shared by the kernels around the recurrences (norm, short convolution) and
// the selective scan: parameter structs, the map from segments to documents, and small device
// helpers.  Not installed.
#pragma once
#include "kda_device.h"

namespace kda {

constexpr int kLayerThreads = 256;   // 4 wave64
// Tokens between the states that the selective backward keeps, whose own states a lane then holds: S x (6 + 1) registers
// at S = 16.  Fewer move more, more spill.  A backward of 4 x 4096 tokens x 4096 channels (bf16, gated), in us:
//     S = 8     4: 866   5: 856   6: 820   7: 846   8: 884   10: 885
//     S = 16    4: 1501  5: 1439  6: 1369  7: 1785
//     S = 32    2: 4558  3: 4137  4: 3872  5: 3765  6: 3852  7: 4312  8: 4967
constexpr int selective_kept(int S) { return S == 32 ? 5 : 6; }

// ---------------------------------------------------------------- norm
struct NormParams {
    const void* x;          // [rows,C]; backward: the stored sum
    const void* residual;   // [rows,C] or nullptr
    const void* weight;     // [C] or nullptr
    void* y;
    void* s;                // [rows,C] or nullptr
    float* scale;           // [rows] (8-bit outputs)
    const void* dy;         // [rows,C]
    const void* ds;         // [rows,C] or nullptr
    void* dx;
    float* dw_part;         // [blocks,C] or nullptr
    int64_t rows;
    int32_t C, out, weight_bf16;   // out: KDA_F32, KDA_BF16, KDA_I8, KDA_E4M3
    float eps;
};

// ---------------------------------------------------------------- convolution
struct ConvParams {
    const void* x;
    const void* weight;     // [C,W]
    const void* bias;       // [C] or nullptr
    const int32_t* cu;
    const void* s0;         // [N,W-1,C] or nullptr
    void* y;
    void* sfinal;           // [N,W-1,C] or nullptr
    const void* dy;
    const void* dsf;        // [N,W-1,C] or nullptr
    void* dx;
    void* ds0;              // [N,W-1,C] or nullptr
    float* part;            // [slots,W+1,C] sums of dweight's taps and dbias
    int64_t T, x_stride;
    int32_t N, C, seqlen, len, slots, out_bf16, weight_bf16, silu, eight;   // eight: channels a thread, else one
};

// ---------------------------------------------------------------- selective scan
struct SelectiveParams {
    const void* x;
    const void* dt;
    const float* A;         // [C,S]
    const void* B;          // [T,G,S]
    const void* Cm;         // [T,G,S]
    const float* D;         // [C] or nullptr
    const void* z;          // [T,C] or nullptr
    const float* bias;      // [C] or nullptr
    const int32_t* cu;
    const float* s0;        // [N,C,S] or nullptr
    void* y;
    float* sfinal;          // [N,C,S] or nullptr
    // segments: own sums, replaced by the entering states; sums of dt
    float* seg;             // [slots,S/4,C,4]
    float* sdt;             // [slots,C]
    // backward
    const void* dy;
    const float* dsf;       // [N,C,S] or nullptr
    float* rseg;            // [slots,S/4,C,4]: likewise from the ends, gradients of the states
    float* border;          // [borders,S/4,C,4] own states before every kept block of tokens
    float* bdt;             // [borders,C] sums of dt up to there
    float* bc_part;         // [T,waves,2,S] a wave's share of dB, dC
    float* par_part;        // [slots,S+2,C] a segment's dA, dD, dbias
    void* dx;
    void* ddt;
    float* dA;
    void* dB;
    void* dC;
    float* dD;
    void* dz;
    float* dbias;
    float* ds0;             // [N,C,S] or nullptr
    int64_t T, x_stride, dt_stride, z_stride, b_stride, c_stride;
    int32_t N, C, G, seqlen, len, slots, out_bf16, softplus, cut, waves, group_waves;   // len: tokens a segment; waves: of 64 channels, group_waves a group
};

// Segments of `len` tokens: segment j of document n has slot floor(start / len) + n + j, so
// every document, empty ones too, has a slot of its own and all lie below T / len + N.
inline int64_t layer_slots(int64_t T, int32_t N, int32_t len) { return T / len + N; }

struct Segment {
    int n, j;                 // document, segment in it
    int64_t lo, hi;           // the document's tokens
    int64_t begin, end;       // the segment's (begin >= end: none)
    bool last;                // the document ends here
};
__device__ __forceinline__ int64_t doc_start(const int32_t* cu, int n, int seqlen, int64_t T) {
    const int64_t x = cu ? (int64_t)cu[n] : (int64_t)n * seqlen;
    return x < 0 ? 0 : x > T ? T : x;
}
// A wave looks for the slot's document 64 at a time: one load for up to 64 documents, two for 4096.
__device__ __forceinline__ Segment find_segment(const int32_t* cu, int N, int seqlen, int64_t T, int len, int64_t slot) {
    int lo = 0, count = N;                    // the document is in [lo, lo + count)
    while (count > 1) {
        const int step = (count + 63) >> 6, at = lo + (int)(threadIdx.x & 63) * step;
        const bool before = at < lo + count && doc_start(cu, at, seqlen, T) / len + at <= slot;
        const int steps = max(__popcll(__ballot(before)) - 1, 0);   // the first holds unless cu_seqlens is malformed
        count = count - steps * step < step ? count - steps * step : step;
        lo += steps * step;
    }
    Segment s;
    s.n = __builtin_amdgcn_readfirstlane(lo);
    s.lo = doc_start(cu, s.n, seqlen, T);
    s.hi = doc_start(cu, s.n + 1, seqlen, T);
    if (s.hi < s.lo) s.hi = s.lo;
    s.j = (int)(slot - (s.lo / len + s.n));
    if (s.j < 0) {                            // malformed
        s.j = 1;
        s.hi = s.lo;
    }
    s.begin = s.lo + (int64_t)s.j * len;
    s.end = s.begin + len < s.hi ? s.begin + len : s.hi;
    s.last = s.end == s.hi && (s.begin < s.end || s.j == 0);
    return s;
}

// x / (1 + e^-x): the exponential of a very negative x is infinite and the quotient 0.
__device__ __forceinline__ float sigmoid_fast(float x) { return __builtin_amdgcn_rcpf(1.f + fast_exp2(-1.44269504f * x)); }

// log(1 + e^v).  With w = 1 + e rounded, log(1 + e) = log(w) + (e - (w - 1)) / w to first order, which keeps every bit of a
// small e.  The quotient may go: w is near 1 where the term counts, and elsewhere it is below half a step of the result.
__device__ __forceinline__ float softplus(float v) {
    const float e = fast_exp2(-1.44269504f * __builtin_fabsf(v)), w = 1.f + e;
    const float l = __builtin_fmaf(__builtin_amdgcn_logf(w), 0.693147181f, e - (w - 1.f));
    return __builtin_fmaxf(v, 0.f) + l;
}

// Eight channels side by side as they lie in memory, at any address: global memory takes 16-byte accesses at the
// alignment of an element.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    typedef bf16x8 __attribute__((aligned(2))) Any;
    bf16x8 r;
    __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const Any*>(p); }
    __device__ __forceinline__ void set(int j, bf16 x) { r[j] = x; }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(r)); }   // waits for the load here
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const f32x4 a = unpack4(__builtin_shufflevector(r, r, 0, 1, 2, 3)), b = unpack4(__builtin_shufflevector(r, r, 4, 5, 6, 7));
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[j + 4] = b[j]; }
    }
};
template <> struct Raw8<float> {
    typedef f32x4 __attribute__((aligned(4))) Any;
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const Any*>(p);
        b = *reinterpret_cast<const Any*>(p + 4);
    }
    __device__ __forceinline__ void set(int j, float x) {
        if (j < 4) a[j] = x;
        else b[j - 4] = x;
    }
    __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(a), "+v"(b)); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[j + 4] = b[j]; }
    }
};
template <typename T> __device__ __forceinline__ void load8(float (&v)[8], const T* p) {
    Raw8<T> x;
    x.load(p);
    x.get(v);
}
// STREAM: a hint that the caches need not keep what is stored, for outputs as large as a prompt's; 16411 rows of 4096
// bf16 channels through the norm take 97 us without and 80 with it.
template <bool STREAM = false> __device__ __forceinline__ void store8_out(void* p, int64_t i, const float (&v)[8], bool as_bf16) {
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    Raw8<bf16>::Any* h = reinterpret_cast<Raw8<bf16>::Any*>((bf16*)p + i);
    Raw8<float>::Any* f = reinterpret_cast<Raw8<float>::Any*>((float*)p + i);
    Raw8<float>::Any* g = reinterpret_cast<Raw8<float>::Any*>((float*)p + i + 4);
    if (as_bf16) {
        if constexpr (STREAM) __builtin_nontemporal_store(pack8<bf16>(a, b), h);
        else *h = pack8<bf16>(a, b);
    } else if constexpr (STREAM) {
        __builtin_nontemporal_store(a, f);
        __builtin_nontemporal_store(b, g);
    } else {
        *f = a;
        *g = b;
    }
}

// Sums of `parts` rows of [K][C] partial sums: rows 0 .. K - 1 of the total go to the arguments in turn, the
// first `taps` of them interleaved as first[c * taps + k].
struct PartSums {
    const float* part;
    int64_t parts;
    int32_t K, C, taps;
    float* first;
    float* rest[2];           // rows taps, taps + 1 (nullptr: dropped)
};
hipError_t launch_part_sums(const PartSums& s, hipStream_t stream);

// Uniform addresses through the scalar cache.
template <typename V> __device__ __forceinline__ V uniform_load(const void* p) {
    typedef const __attribute__((address_space(4))) V* P;
    return *(P)(uintptr_t)p;
}

__device__ __forceinline__ void store_out(void* p, int64_t i, float x, bool as_bf16) {
    if (as_bf16) ((bf16*)p)[i] = (bf16)x;
    else ((float*)p)[i] = x;
}

// The forward's rows a workgroup and its threads.
inline int norm_fwd_rows(int32_t C) { return C <= 128 ? 16 : C <= 256 ? 8 : C <= 1024 ? 4 : 1; }
inline int norm_fwd_threads(int32_t C) { return C <= 8192 ? kLayerThreads : 512; }
hipError_t launch_norm_fwd(const NormParams& p, int in_bf16, int res_bf16, hipStream_t stream);
hipError_t launch_norm_bwd(const NormParams& p, int in_bf16, int res_bf16, float* dw, hipStream_t stream);
int norm_bwd_blocks(int32_t C, int64_t rows);
hipError_t launch_conv_fwd(const ConvParams& p, int W, int in_bf16, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvParams& p, int W, int in_bf16, float* dw, float* db, hipStream_t stream);
hipError_t launch_conv_decode(const ConvParams& p, int W, int in_bf16, hipStream_t stream);
hipError_t launch_selective_states(const SelectiveParams& p, int S, int in_bf16, bool backward, hipStream_t stream);
hipError_t launch_selective_out(const SelectiveParams& p, int S, int in_bf16, hipStream_t stream);
hipError_t launch_selective_grads(const SelectiveParams& p, int S, int in_bf16, hipStream_t stream);
hipError_t launch_selective_decode(const SelectiveParams& p, int S, int in_bf16, hipStream_t stream);

}  // namespace kda
