// kda_norm.hip -- root-mean-square norm of rows with the residual's addition, in the input's
// type or in 8 bits, and its backward:
//     s = x + residual,  y = s w rstd,  rstd = 1 / sqrt(mean(s^2) + eps)
//     dx = rstd (w dy - s rstd^2 mean(w dy s)) + ds,  dw = sum over rows of dy s rstd
// A row is read once into registers, summed across its lanes, and written: the bytes bound it.
#include "kda_layer.h"

namespace kda {

// Columns of a thread: i-th group of eight side by side (VEC), or all of them TPR apart.
template <int TPR, bool VEC> __device__ __forceinline__ int norm_col(int tid, int i, int j) {
    return VEC ? (tid + TPR * i) * 8 + j : tid + TPR * (8 * i + j);
}
template <typename T, int TPR, int NC, bool VEC>
__device__ __forceinline__ void norm_load(float (&v)[NC][8], const T* row, int tid, int C) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if constexpr (VEC) {
            const int c = norm_col<TPR, VEC>(tid, i, 0);
            if (c < C) load8(v[i], row + c);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = norm_col<TPR, VEC>(tid, i, j);
                v[i][j] = c < C ? to_f32(row[c]) : 0.f;
            }
        }
    }
}
template <int TPR, bool VEC>
__device__ __forceinline__ void norm_store(void* base, int64_t at, int tid, int i, int C, const float (&v)[8], bool as_bf16) {
    if constexpr (VEC) {
        const int c = norm_col<TPR, VEC>(tid, i, 0);
        if (c < C) store8_out(base, at + c, v, as_bf16);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = norm_col<TPR, VEC>(tid, i, j);
            if (c < C) store_out(base, at + c, v[j], as_bf16);
        }
    }
}
template <int TPR, bool VEC>
__device__ __forceinline__ void norm_weight(float (&w)[8], const NormParams& p, int tid, int i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    if (!p.weight) return;
    if constexpr (VEC) {
        const int c = norm_col<TPR, VEC>(tid, i, 0);
        if (c >= p.C) return;
        if (p.weight_bf16) load8(w, (const bf16*)p.weight + c);
        else load8(w, (const float*)p.weight + c);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = norm_col<TPR, VEC>(tid, i, j);
            if (c < p.C) w[j] = p.weight_bf16 ? to_f32(((const bf16*)p.weight)[c]) : ((const float*)p.weight)[c];
        }
    }
}

// Over the TPR threads of a row, the same value in each; `red` holds one value a wave.
template <int TPR, typename V, typename F> __device__ __forceinline__ V row_reduce(V x, V* red, F f) {
#pragma unroll
    for (int m = 32; m; m >>= 1) x = f(x, __shfl_xor(x, m, 64));
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

// mean(s^2) may leave fp32's range where s does not: such rows are summed again scaled by a power of two.
template <int TPR, int NC> __device__ __forceinline__ float norm_rstd(const float (&v)[NC][8], const NormParams& p, float* red) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(v[i][j], v[i][j], sum);
    sum = row_reduce<TPR>(sum, red, Add());
    if (__builtin_expect(!(sum < __builtin_huge_valf()), 0)) {
        constexpr float k = 0x1p-80f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(v[i][j] * k, v[i][j] * k, sum);
        sum = row_reduce<TPR>(sum, red, Add());
        return k / sqrtf(sum / (float)p.C);      // eps is far below such a mean
    }
    return 1.f / sqrtf(sum / (float)p.C + p.eps);
}

template <typename TI, typename TR, int TPR, int NC, bool VEC>
__global__ __launch_bounds__(TPR < kLayerThreads ? kLayerThreads : TPR) void norm_fwd_kernel(NormParams p) {
    constexpr int RPB = TPR < kLayerThreads ? kLayerThreads / TPR : 1;
    __shared__ float red[TPR / 64];
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (row >= p.rows) return;                   // whole waves: a row of several waves is a workgroup of its own
    const int64_t at = row * p.C;
    float v[NC][8];
    norm_load<TI, TPR, NC, VEC>(v, (const TI*)p.x + at, tid, p.C);
    if (p.residual) {
        float r[NC][8];
        norm_load<TR, TPR, NC, VEC>(r, (const TR*)p.residual + at, tid, p.C);
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = to_f32(from_f32<TR>(v[i][j] + r[i][j]));
        if (p.s)
#pragma unroll
            for (int i = 0; i < NC; ++i) norm_store<TPR, VEC>(p.s, at, tid, i, p.C, v[i], sizeof(TR) == 2);
    }
    const float rstd = norm_rstd<TPR>(v, p, red);
    if (p.out < 2) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float w[8];
            norm_weight<TPR, VEC>(w, p, tid, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] *= rstd * w[j];
            norm_store<TPR, VEC>(p.y, at, tid, i, p.C, v[i], p.out == 1);
        }
        return;
    }
    unsigned top = 0;                            // of the products' absolute values as bits: NaN is above all others
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float w[8];
        norm_weight<TPR, VEC>(w, p, tid, i);
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
    if (tid == 0) p.scale[row] = top < 0x7f800000u ? amax * rstd / Q : __builtin_nanf("");
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
        if constexpr (VEC) {
            const int c = norm_col<TPR, VEC>(tid, i, 0);
            const u32x2 both = {word[0], word[1]};
            if (c < p.C) *reinterpret_cast<u32x2*>(y + c) = both;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = norm_col<TPR, VEC>(tid, i, j);
                if (c < p.C) y[c] = (uint8_t)(word[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
}

// A workgroup goes over rows gridDim apart and keeps its sums for dw in registers.
template <typename TI, typename TR, int TPR, int NC, bool VEC>
__global__ __launch_bounds__(TPR < kLayerThreads ? kLayerThreads : TPR) void norm_bwd_kernel(NormParams p) {
    constexpr int RPB = TPR < kLayerThreads ? kLayerThreads / TPR : 1;
    __shared__ float red[TPR / 64];
    const int tid = threadIdx.x % TPR;
    const int64_t first = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR, step = (int64_t)gridDim.x * RPB;
    float acc[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    for (int64_t row = first; row < p.rows; row += step) {
        const int64_t at = row * p.C;
        float v[NC][8], g[NC][8];
        norm_load<TR, TPR, NC, VEC>(v, (const TR*)p.x + at, tid, p.C);
        norm_load<TI, TPR, NC, VEC>(g, (const TI*)p.dy + at, tid, p.C);
        const float rstd = norm_rstd<TPR>(v, p, red);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float w[8];
            norm_weight<TPR, VEC>(w, p, tid, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= rstd;
                acc[i][j] = __builtin_fmaf(g[i][j], v[i][j], acc[i][j]);
                g[i][j] *= w[j];
                dot = __builtin_fmaf(g[i][j], v[i][j], dot);
            }
        }
        const float mean = row_reduce<TPR>(dot, red, Add()) / (float)p.C;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = rstd * (g[i][j] - v[i][j] * mean);
        }
        if (p.ds) {
            norm_load<TR, TPR, NC, VEC>(g, (const TR*)p.ds + at, tid, p.C);
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += g[i][j];
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) norm_store<TPR, VEC>(p.dx, at, tid, i, p.C, v[i], p.out == 1);
    }
    if (p.dw_part)
#pragma unroll
        for (int i = 0; i < NC; ++i) norm_store<TPR, VEC>(p.dw_part, first * p.C, tid, i, p.C, acc[i], false);
}

// One workgroup for 64 columns: 16 waves take every 16th row, then their sums in order.
__global__ __launch_bounds__(1024) void part_sums_kernel(PartSums s) {
    __shared__ float sum[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t cols = (int64_t)s.K * s.C, col = (int64_t)blockIdx.x * 64 + lane;
    float x = 0.f;
    if (col < cols)
#pragma unroll 8
        for (int64_t r = w; r < s.parts; r += 16) x += s.part[r * cols + col];
    sum[w][lane] = x;
    __syncthreads();
    if (w || col >= cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) x += sum[i][lane];
    const int k = (int)(col / s.C), c = (int)(col % s.C);
    if (k < s.taps) s.first[(int64_t)c * s.taps + k] = x;
    else if (s.rest[k - s.taps]) s.rest[k - s.taps][c] = x;
}
hipError_t launch_part_sums(const PartSums& s, hipStream_t stream) {
    const int64_t cols = (int64_t)s.K * s.C;
    hipLaunchKernelGGL(part_sums_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, stream, s);
    return hipGetLastError();
}

// ---------------------------------------------------------------- launches
template <typename TI, typename TR, int TPR, int NC, bool VEC>
static void norm_launch(const NormParams& p, bool backward, int blocks, hipStream_t stream) {
    constexpr int threads = TPR < kLayerThreads ? kLayerThreads : TPR, RPB = threads / TPR;
    if (backward) hipLaunchKernelGGL((norm_bwd_kernel<TI, TR, TPR, NC, VEC>), dim3((unsigned)blocks), dim3(threads), 0, stream, p);
    else hipLaunchKernelGGL((norm_fwd_kernel<TI, TR, TPR, NC, VEC>), dim3((unsigned)((p.rows + RPB - 1) / RPB)), dim3(threads), 0, stream, p);
}
template <typename TI, typename TR, bool VEC>
static void norm_size(const NormParams& p, bool backward, int blocks, hipStream_t stream) {
    const int C = p.C;
    if (C <= 512) norm_launch<TI, TR, 64, 1, VEC>(p, backward, blocks, stream);
    else if (C <= 1024) norm_launch<TI, TR, 64, 2, VEC>(p, backward, blocks, stream);
    else if (C <= 2048) norm_launch<TI, TR, 256, 1, VEC>(p, backward, blocks, stream);
    else if (C <= 4096) norm_launch<TI, TR, 256, 2, VEC>(p, backward, blocks, stream);
    else if (C <= 8192) norm_launch<TI, TR, 256, 4, VEC>(p, backward, blocks, stream);
    else if (C <= 16384) norm_launch<TI, TR, 512, 4, VEC>(p, backward, blocks, stream);
    else norm_launch<TI, TR, 512, 8, VEC>(p, backward, blocks, stream);
}
template <typename TI, typename TR> static void norm_vec(const NormParams& p, bool backward, int blocks, hipStream_t stream) {
    if (p.C % 8 == 0) norm_size<TI, TR, true>(p, backward, blocks, stream);
    else norm_size<TI, TR, false>(p, backward, blocks, stream);
}
static hipError_t norm_any(const NormParams& p, int in_bf16, int res_bf16, bool backward, int blocks, hipStream_t stream) {
    if (in_bf16 && res_bf16) norm_vec<bf16, bf16>(p, backward, blocks, stream);
    else if (in_bf16) norm_vec<bf16, float>(p, backward, blocks, stream);
    else norm_vec<float, float>(p, backward, blocks, stream);
    return hipGetLastError();
}
hipError_t launch_norm_fwd(const NormParams& p, int in_bf16, int res_bf16, hipStream_t stream) {
    return norm_any(p, in_bf16, res_bf16, false, 0, stream);
}

// Rows of partial sums of dw: one a row's worth of threads of every workgroup.
static int norm_rows_at_once(int32_t C) { return C <= 1024 ? 4 : 1; }
int norm_bwd_blocks(int32_t C, int64_t rows) {
    const int64_t groups = (rows + norm_rows_at_once(C) - 1) / norm_rows_at_once(C);
    return (int)(groups < 1024 ? groups : 1024);
}
int64_t norm_bwd_parts(int32_t C, int64_t rows) { return (int64_t)norm_bwd_blocks(C, rows) * norm_rows_at_once(C); }
hipError_t launch_norm_bwd(const NormParams& p, int in_bf16, int res_bf16, float* dw, hipStream_t stream) {
    if (p.rows) {
        const hipError_t e = norm_any(p, in_bf16, res_bf16, true, norm_bwd_blocks(p.C, p.rows), stream);
        if (e != hipSuccess) return e;
    }
    if (!dw) return hipSuccess;
    const PartSums s = {p.dw_part, norm_bwd_parts(p.C, p.rows), 1, p.C, 1, dw, {nullptr, nullptr}};
    return launch_part_sums(s, stream);
}

}  // namespace kda
