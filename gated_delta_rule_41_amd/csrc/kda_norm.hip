// kda_norm.hip -- root-mean-square norm of rows with the residual's addition, in the input's
// type or in 8 bits, and its backward:
//     s = x + residual,  y = s w rstd,  rstd = 1 / sqrt(mean(s^2) + eps)
//     dx = rstd (w dy - s rstd^2 mean(w dy s)) + ds,  dw = sum over rows of dy s rstd
// A row is read once into registers, summed across its lanes, and written: the bytes bound it.
// bf16, with a residual, 16411 x 4096 take 76 us (7.1 TB/s, the last cache's share in it), the
// backward of 32768 x 4096 193 (5.6 TB/s).
#include "kda_layer.h"

namespace kda {

// A thread's i-th eight channels begin at (tid + TPR i) 8; a row's last eight may be fewer.  Every thread loads eight
// channels, the row's last ones where its own are not all there, and puts them right when they have come.  kEarly, for rows
// asked for early: threads behind the row load too, as zeros written in a branch beside a load wait for that load (backward
// of 26214 x 2560 187 us so, 119 without; 209715 x 320 176 and 104).  kHere: where nothing is early they load nothing
// (forward of 52428 x 1280 90, and 94 if they do).  kShort: early rows of fewer than eight channels, which have no eight to
// load, element by element.
enum NormWay { kHere, kEarly, kShort };
template <int TPR> __device__ __forceinline__ int norm_col(int tid, int i) { return (tid + TPR * i) * 8; }
template <typename T, int WAY> struct NormEight : Raw8<T> {
    __device__ __forceinline__ void ask(const T* row, int c, int C) {
        if constexpr (WAY == kShort) {
#pragma unroll
            for (int j = 0; j < 8; ++j) this->set(j, row[c + j < C ? c + j : 0]);
        } else if (WAY == kEarly || (c < C && C >= 8)) {
            this->load(row + (c + 8 <= C ? c : C - 8));
        }
    }
    __device__ __forceinline__ void take(float (&v)[8], const T* row, int c, int C) const {
        this->get(v);
        if (WAY != kShort && c + 8 <= C) return;
        if (WAY == kHere && C < 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f32(row[j < C ? j : 0]);
        } else if (WAY != kShort) {
            const int by = 8 - (C & 7);           // the same for the whole row's end; 8: a row of whole pieces
#pragma unroll
            for (int m = 4; m; m >>= 1)
                if (by & m)
#pragma unroll
                    for (int j = 0; j + m < 8; ++j) v[j] = v[j + m];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c + j < C ? v[j] : 0.f;
    }
};
template <typename T> __device__ __forceinline__ void norm_load8(float (&v)[8], const T* row, int c, int C) {
    NormEight<T, kHere> r;
    r.ask(row, c, C);
    r.take(v, row, c, C);
}
// A row's groups as they lie in memory, to be asked for early.
template <typename T, int TPR, int NC, int WAY> struct NormRow {
    NormEight<T, WAY> r[NC];
    __device__ __forceinline__ void load(const T* row, int tid, int C) {
#pragma unroll
        for (int i = 0; i < NC; ++i) r[i].ask(row, norm_col<TPR>(tid, i), C);
    }
    __device__ __forceinline__ void get(float (&v)[NC][8], const T* row, int tid, int C) const {
#pragma unroll
        for (int i = 0; i < NC; ++i) r[i].take(v[i], row, norm_col<TPR>(tid, i), C);
    }
};
__device__ __forceinline__ void norm_store8(void* base, int64_t at, int c, int C, const float (&v)[8], bool as_bf16) {
    if (c + 8 <= C) {
        store8_out<true>(base, at + c, v, as_bf16);
    } else if (c < C) {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (c + j < C) store_out(base, at + c + j, v[j], as_bf16);
    }
}
// Fewer than eight weights in fp32 by constant indexes, each behind its own test: at j < C ? j : 0, the same for all lanes,
// this compiler made scalar loads with half of the byte offset in the base, where bf16 has all of it, and half in the
// index, and a scalar load drops the two lowest bits of each, so that elements 1, 3 and 5 were their neighbours.  (bf16
// has no scalar loads; by tests the forward of 1048576 x 7 takes 103 us, 91 without.)
template <typename T> __device__ __forceinline__ void norm_weight(float (&w)[8], const NormParams& p, int c) {
    const T* weight = (const T*)p.weight;
    if (sizeof(T) == 2 || p.C >= 8) {
        norm_load8(w, weight, c, p.C);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = 0.f;
            if (c + j < p.C) w[j] = to_f32(weight[j]);   // c is 0
        }
    }
}
__device__ __forceinline__ void norm_weight(float (&w)[8], const NormParams& p, int c) {
    if (!p.weight) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 1.f;
    } else if (p.weight_bf16) {
        norm_weight<bf16>(w, p, c);
    } else {
        norm_weight<float>(w, p, c);
    }
}

// Over the TPR threads of a row, the same value in each; `red` holds one value a wave.
template <int TPR, typename V, typename F> __device__ __forceinline__ V row_reduce(V x, V* red, F f) {
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m; m >>= 1) x = f(x, __shfl_xor(x, m, 64));
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w) x = f(x, red[w]);
    }
    return x;
}

struct Add { __device__ float operator()(float a, float b) const { return a + b; } };
struct MaxBits { __device__ unsigned operator()(unsigned a, unsigned b) const { return a > b ? a : b; } };

// p Q / m in 24 bits and rounded to odd: any later rounding to fewer bits then gives the nearest
// value, ties to even, as if from the exact quotient.  m in [0.5, 1), inv ~ 1 / m.
__device__ __forceinline__ float odd_quotient(float p, float Q, float m, float inv) {
    const float h = p * Q, l = __builtin_fmaf(p, Q, -h);
    const float q0 = h * inv;
    const float q = __builtin_fmaf(__builtin_fmaf(-q0, m, h) + l, inv, q0);
    const float r = __builtin_fmaf(-q, m, h) + l;   // what q leaves; its sign is exact
    unsigned b = __float_as_uint(q);
    if (r != 0.f && q != 0.f && !(b & 1)) b += (r > 0.f) == (q > 0.f) ? 1u : ~0u;
    return __uint_as_float(b);
}

// mean(s^2) may leave fp32's range, or the part of it where squares keep their bits, though s does not: such rows are
// summed again, scaled by a power of two.  The normed row is then s by rstd.
struct NormScale { float rstd, by; };
__device__ __forceinline__ float norm_scale_by(float mean_eps) {
    if (__builtin_expect(mean_eps >= 0x1p-96f && mean_eps < __builtin_huge_valf(), 1)) return 1.f;
    return mean_eps < 1.f ? 0x1p100f : 0x1p-80f;
}
__device__ __forceinline__ float norm_mean_eps(float sum, const NormParams& p, float by) { return sum / (float)p.C + p.eps * by * by; }
template <int NC> __device__ __forceinline__ void norm_scale(float (&v)[NC][8], float by) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= by;
}
template <int TPR, int NC> __device__ __forceinline__ NormScale norm_rstd(const float (&v)[NC][8], const NormParams& p, float* red) {
    auto mean = [&](float by) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(v[i][j] * by, v[i][j] * by, sum);
        return norm_mean_eps(row_reduce<TPR>(sum, red, Add()), p, by);
    };
    float m = mean(1.f);
    const float by = norm_scale_by(m);
    if (by != 1.f) m = mean(by);
    return {1.f / sqrtf(m), by};
}

template <typename TI, typename TR, int TPR, int NC>
__global__ __launch_bounds__(TPR < kLayerThreads ? kLayerThreads : TPR) void norm_fwd_kernel(NormParams p) {
    constexpr int RPB = TPR < kLayerThreads ? kLayerThreads / TPR : 1;
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (row >= p.rows) return;                   // a row of several waves is a workgroup of its own
    const int64_t at = row * p.C;
    float v[NC][8];
    NormRow<TI, TPR, NC, kHere> x;
    NormRow<TR, TPR, NC, kHere> res;
    x.load((const TI*)p.x + at, tid, p.C);
    if (p.residual) res.load((const TR*)p.residual + at, tid, p.C);
    x.get(v, (const TI*)p.x + at, tid, p.C);
    if (p.residual) {
        float r[NC][8];
        res.get(r, (const TR*)p.residual + at, tid, p.C);
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = to_f32(from_f32<TR>(v[i][j] + r[i][j]));
        if (p.s)
#pragma unroll
            for (int i = 0; i < NC; ++i) norm_store8(p.s, at, norm_col<TPR>(tid, i), p.C, v[i], sizeof(TR) == 2);
    }
    const NormScale n = norm_rstd<TPR>(v, p, red);
    if (p.out < 2) {
        if (n.by != 1.f) norm_scale(v, n.by);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float w[8];
            norm_weight(w, p, norm_col<TPR>(tid, i));
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= n.rstd * w[j];
            norm_store8(p.y, at, norm_col<TPR>(tid, i), p.C, v[i], p.out == 1);
        }
        return;
    }
    unsigned top = 0;                            // of the products' absolute values as bits: NaN is above all others
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float w[8];
        norm_weight(w, p, norm_col<TPR>(tid, i));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] *= w[j];
            const unsigned b = __float_as_uint(v[i][j]) & 0x7fffffffu;
            top = b > top ? b : top;
        }
    }
    top = row_reduce<TPR>(top, reinterpret_cast<unsigned*>(red), MaxBits());
    const float amax = __uint_as_float(top), Q = p.out == 2 ? 127.f : 448.f;
    const bool codes = top != 0 && top < 0x7f800000u;
    if (tid == 0) p.scale[row] = codes ? amax * n.by * n.rstd / Q : top == 0 ? 0.f : __builtin_nanf("");
    const int e = codes ? __builtin_amdgcn_frexp_expf(amax) : 0;
    const float m = codes ? __builtin_amdgcn_ldexpf(amax, -e) : 1.f, inv = __builtin_amdgcn_rcpf(m);
    uint8_t* y = (uint8_t*)p.y + at;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        unsigned word[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float a = odd_quotient(__builtin_amdgcn_ldexpf(v[i][j], -e), Q, m, inv);
            const float b = odd_quotient(__builtin_amdgcn_ldexpf(v[i][j + 1], -e), Q, m, inv);
            unsigned pair;
            if (p.out == 2) pair = ((unsigned)(int)__builtin_rintf(a) & 255u) | (((unsigned)(int)__builtin_rintf(b) & 255u) << 8);
            else pair = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xffffu;
            word[j >> 2] |= pair << (8 * (j & 2));
        }
        if (!codes) word[0] = word[1] = 0;
        const int c = norm_col<TPR>(tid, i);
        if (c + 8 <= p.C) {
            typedef u32x2 __attribute__((aligned(1))) codes8;
            __builtin_nontemporal_store(u32x2{word[0], word[1]}, reinterpret_cast<codes8*>(y + c));
        } else if (c < p.C) {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (c + j < p.C) y[c + j] = (uint8_t)(word[j >> 2] >> (8 * (j & 3)));
        }
    }
}

struct Sums { float square, dot; };
struct AddSums { __device__ Sums operator()(Sums a, Sums b) const { return {a.square + b.square, a.dot + b.dot}; } };
template <int TPR> __device__ __forceinline__ Sums row_sums(Sums x, Sums* red) {
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m; m >>= 1) x = AddSums()(x, {__shfl_xor(x.square, m, 64), __shfl_xor(x.dot, m, 64)});
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int w = 1; w < W; ++w) x = AddSums()(x, red[w]);
    }
    return x;
}

// dx = rstd (w dy - s rstd^2 mean(w dy s)) + ds: both sums of a row come from one pass over it.  A workgroup goes over
// rows gridDim apart and keeps its sums for dw in registers.  Up to three groups of eight channels a thread stay there as
// well, the weights too, with the next row's s and dy on their way, which have to be there before this row's dx is
// stored: a later wait for them would be one for the stores as well (209715 x 320 bf16 162 -> 143 us).  Rows above 12288
// channels are read again from the caches.
template <typename TI, typename TR, int TPR, int NC, int WAY>
__global__ __launch_bounds__(TPR < kLayerThreads ? kLayerThreads : TPR) void norm_bwd_kernel(NormParams p) {
    constexpr int RPB = TPR < kLayerThreads ? kLayerThreads / TPR : 1;
    constexpr bool kHeld = TPR <= 512;
    static_assert(!kHeld || NC <= 3, "a held row has up to three groups a thread");
    constexpr int H = kHeld ? NC : 1;
    __shared__ Sums red[TPR > 64 ? TPR / 64 : 1];
    const int tid = threadIdx.x % TPR;
    const int64_t first = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR, step = (int64_t)gridDim.x * RPB;
    float acc[NC][8], w[H][8], v[H][8], g[H][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    NormRow<TR, TPR, H, WAY> ns, nds;
    NormRow<TI, TPR, H, WAY> ng;
    if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < NC; ++i) norm_weight(w[i], p, norm_col<TPR>(tid, i));
        if (first < p.rows) {
            ns.load((const TR*)p.x + first * p.C, tid, p.C);
            ng.load((const TI*)p.dy + first * p.C, tid, p.C);
        }
    }
    for (int64_t row = first; row < p.rows; row += step) {
        const int64_t at = row * p.C;
        const TR* s = (const TR*)p.x + at;
        const TI* dy = (const TI*)p.dy + at;
        if constexpr (kHeld) {
            ns.get(v, s, tid, p.C);
            ng.get(g, dy, tid, p.C);
            if (p.ds) nds.load((const TR*)p.ds + at, tid, p.C);
            if (row + step < p.rows) {
                ns.load(s + step * p.C, tid, p.C);
                ng.load(dy + step * p.C, tid, p.C);
            }
        }
        float by = 1.f;
        auto group = [&](int i) {                 // s, dy and the weights of the i-th group, in v, g, w[h]
            if constexpr (!kHeld) {
                const int c = norm_col<TPR>(tid, i);
                norm_load8(v[0], s, c, p.C);
                if (by != 1.f) norm_scale(v, by);
                norm_load8(g[0], dy, c, p.C);
                norm_weight(w[0], p, c);
            }
            return kHeld ? i : 0;
        };
        auto sums = [&]() {
            Sums x = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int h = group(i);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x.square = __builtin_fmaf(v[h][j], v[h][j], x.square);
                    x.dot = __builtin_fmaf(w[h][j] * g[h][j], v[h][j], x.dot);
                }
            }
            return row_sums<TPR>(x, red);
        };
        Sums x = sums();
        by = norm_scale_by(norm_mean_eps(x.square, p, 1.f));
        if (by != 1.f) {
            if constexpr (kHeld) norm_scale(v, by);
            x = sums();
        }
        const float rstd = 1.f / sqrtf(norm_mean_eps(x.square, p, by));
        const float mean = x.dot * rstd / (float)p.C;       // of w dy and the normed row
        const float slope = rstd * by;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int h = group(i), c = norm_col<TPR>(tid, i);
            float (&dx)[8] = kHeld ? v[h] : v[0], e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = v[h][j] * rstd;
                acc[i][j] = __builtin_fmaf(g[h][j], xh, acc[i][j]);
                dx[j] = slope * (w[h][j] * g[h][j] - xh * mean);
            }
            if (p.ds) {
                if constexpr (kHeld) nds.r[i].take(e, (const TR*)p.ds + at, c, p.C);
                else norm_load8(e, (const TR*)p.ds + at, c, p.C);
#pragma unroll
                for (int j = 0; j < 8; ++j) dx[j] += e[j];
            }
            if constexpr (!kHeld) norm_store8(p.dx, at, c, p.C, dx, p.out == 1);
        }
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < NC; ++i) { ns.r[i].arrived(); ng.r[i].arrived(); }
#pragma unroll
            for (int i = 0; i < NC; ++i) norm_store8(p.dx, at, norm_col<TPR>(tid, i), p.C, v[i], p.out == 1);
        }
    }
    if (!p.dw_part) return;
    if constexpr (RPB > 1) {                      // the workgroup's rows together: over a wave's lanes, then its waves in order
        __shared__ float waves[kLayerThreads / 64][TPR * NC * 8];
        const int wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int m = TPR; m < 64; m <<= 1) acc[i][j] += __shfl_xor(acc[i][j], m, 64);
                if ((threadIdx.x & 63) < TPR) waves[wave][(i * 8 + j) * TPR + tid] = acc[i][j];
            }
        __syncthreads();
        if (threadIdx.x >= TPR) return;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int w = 1; w < kLayerThreads / 64; ++w) acc[i][j] += waves[w][(i * 8 + j) * TPR + tid];
            }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) norm_store8(p.dw_part, (int64_t)blockIdx.x * p.C, norm_col<TPR>(tid, i), p.C, acc[i], false);
}

// One workgroup for COLS columns: its 1024 / COLS rows of threads take every so many rows, then their sums: over a wave's
// lanes, and its waves in order.
template <int COLS> __global__ __launch_bounds__(1024) void part_sums_kernel(PartSums s) {
    constexpr int ROWS = 1024 / COLS;
    __shared__ float sum[16][COLS];
    const int lane = threadIdx.x % COLS, w = threadIdx.x >> 6;
    const int64_t cols = (int64_t)s.K * s.C, col = (int64_t)blockIdx.x * COLS + lane;
    float x = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int64_t r = threadIdx.x / COLS; r < s.parts; r += ROWS) x += s.part[r * cols + col];
#pragma unroll
    for (int m = COLS; m < 64; m <<= 1) x += __shfl_xor(x, m, 64);
    if ((threadIdx.x & 63) < COLS) sum[w][lane] = x;
    __syncthreads();
    if (threadIdx.x >= COLS || col >= cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) x += sum[i][lane];
    const int k = (int)(col / s.C), c = (int)(col % s.C);
    if (k < s.taps) s.first[(int64_t)c * s.taps + k] = x;
    else if (s.rest[k - s.taps]) s.rest[k - s.taps][c] = x;
}
hipError_t launch_part_sums(const PartSums& s, hipStream_t stream) {
    const int64_t cols = (int64_t)s.K * s.C;
    // Few columns take more workgroups of narrower pieces.  us for 16 and 64 columns a workgroup: 128 columns of 1024
    // parts 4.6 and 6.9, 4096 of 512 5.0 and 5.2, 9216 of 256 4.5 and 3.8, 73728 of 171 25.1 and 13.7.
    if (cols > 4096) hipLaunchKernelGGL((part_sums_kernel<64>), dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, stream, s);
    else hipLaunchKernelGGL((part_sums_kernel<16>), dim3((unsigned)((cols + 15) / 16)), dim3(1024), 0, stream, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------- launches
// A row's threads and groups of eight channels a thread: few threads without channels, and in the backward, which keeps
// five values a channel and rows on their way, up to 24 channels each.  bf16, 2^26 values: 1280 channels 104 us with 64
// threads and three groups, 139 with 192 and one; 5120: 102 with 256 and three, 112 with 320 and two; 12288: 183 with 1024
// and two, read again.
template <typename TI, typename TR, int TPR, int NC> static void norm_fwd_launch(const NormParams& p, hipStream_t stream) {
    constexpr int threads = TPR < kLayerThreads ? kLayerThreads : TPR, RPB = threads / TPR;
    hipLaunchKernelGGL((norm_fwd_kernel<TI, TR, TPR, NC>), dim3((unsigned)((p.rows + RPB - 1) / RPB)), dim3(threads), 0, stream, p);
}
template <typename TI, typename TR, int TPR, int NC, int WAY = kEarly> static void norm_bwd_launch(const NormParams& p, hipStream_t stream) {
    constexpr int threads = TPR < kLayerThreads ? kLayerThreads : TPR;
    hipLaunchKernelGGL((norm_bwd_kernel<TI, TR, TPR, NC, WAY>), dim3((unsigned)norm_bwd_blocks(p.C, p.rows)), dim3(threads), 0, stream, p);
}
template <typename TI, typename TR> static void norm_types(const NormParams& p, bool backward, hipStream_t stream) {
    const int C = p.C;
    if (backward) {
        if (C < 8) norm_bwd_launch<TI, TR, 16, 1, kShort>(p, stream);
        else if (C <= 128) norm_bwd_launch<TI, TR, 16, 1>(p, stream);
        else if (C <= 256) norm_bwd_launch<TI, TR, 32, 1>(p, stream);
        else if (C <= 384) norm_bwd_launch<TI, TR, 16, 3>(p, stream);
        else if (C <= 512) norm_bwd_launch<TI, TR, 64, 1>(p, stream);
        else if (C <= 768) norm_bwd_launch<TI, TR, 32, 3>(p, stream);
        else if (C <= 1024) norm_bwd_launch<TI, TR, 64, 2>(p, stream);
        else if (C <= 1536) norm_bwd_launch<TI, TR, 64, 3>(p, stream);
        else if (C <= 2048) norm_bwd_launch<TI, TR, 256, 1>(p, stream);
        else if (C <= 4096) norm_bwd_launch<TI, TR, 256, 2>(p, stream);
        else if (C <= 6144) norm_bwd_launch<TI, TR, 256, 3>(p, stream);
        else if (C <= 8192) norm_bwd_launch<TI, TR, 512, 2>(p, stream);
        else if (C <= 12288) norm_bwd_launch<TI, TR, 512, 3>(p, stream);
        else norm_bwd_launch<TI, TR, 1024, 2>(p, stream);
    } else {
        if (C <= 128) norm_fwd_launch<TI, TR, 16, 1>(p, stream);
        else if (C <= 256) norm_fwd_launch<TI, TR, 32, 1>(p, stream);
        else if (C <= 512) norm_fwd_launch<TI, TR, 64, 1>(p, stream);
        else if (C <= 1024) norm_fwd_launch<TI, TR, 64, 2>(p, stream);
        else if (C <= 2048) norm_fwd_launch<TI, TR, 256, 1>(p, stream);
        else if (C <= 4096) norm_fwd_launch<TI, TR, 256, 2>(p, stream);
        else if (C <= 8192) norm_fwd_launch<TI, TR, 256, 4>(p, stream);
        else norm_fwd_launch<TI, TR, 512, 4>(p, stream);
    }
}
static hipError_t norm_any(const NormParams& p, int in_bf16, int res_bf16, bool backward, hipStream_t stream) {
    if (in_bf16 && res_bf16) norm_types<bf16, bf16>(p, backward, stream);
    else if (in_bf16) norm_types<bf16, float>(p, backward, stream);
    else norm_types<float, float>(p, backward, stream);
    return hipGetLastError();
}
hipError_t launch_norm_fwd(const NormParams& p, int in_bf16, int res_bf16, hipStream_t stream) {
    return norm_any(p, in_bf16, res_bf16, false, stream);
}

// Workgroups, each with one row of partial sums of dw: as many as the compute units hold at once, so that all go over as
// many rows.  bf16, 2^26 values, us for 1, 2, 3, 4 on a compute unit:  128 channels 300, 176, 136, 121 (100 channels);
// 200: 213, 127, 110, 145;  384: 115, 103, 116, 107;  512: 171, 112, 100, 121;  768: 115, 104, 115, 107;  1000: 145, 101,
// 119, 107;  1280: 139, 104, 121, 107;  2048: 148, 112, 101, 122;  4096: 111, 101, 115, 107;  5120: 122, 102, 119, 108;
// 8192: 98, 102, 106, 113.  Moving the bytes takes 104 at a large copy's rate.
static int norm_rows_at_once(int32_t C) { return C <= 128 ? 16 : C <= 256 ? 8 : C <= 384 ? 16 : C <= 512 ? 4 : C <= 768 ? 8 : C <= 1536 ? 4 : 1; }
int norm_bwd_blocks(int32_t C, int64_t rows) {
    const int64_t groups = (rows + norm_rows_at_once(C) - 1) / norm_rows_at_once(C);
    const int64_t most = 256 * (C <= 128 ? 4 : C <= 256 ? 3 : C <= 384 ? 2 : C <= 512 ? 3 : C <= 1536 ? 2 : C <= 2048 ? 3 : C <= 6144 ? 2 : 1);
    return (int)(groups < most ? groups : most);
}
hipError_t launch_norm_bwd(const NormParams& p, int in_bf16, int res_bf16, float* dw, hipStream_t stream) {
    if (p.rows) {
        const hipError_t e = norm_any(p, in_bf16, res_bf16, true, stream);
        if (e != hipSuccess) return e;
    }
    if (!dw) return hipSuccess;
    const PartSums s = {p.dw_part, norm_bwd_blocks(p.C, p.rows), 1, p.C, 1, dw, {nullptr, nullptr}};
    return launch_part_sums(s, stream);
}

}  // namespace kda
