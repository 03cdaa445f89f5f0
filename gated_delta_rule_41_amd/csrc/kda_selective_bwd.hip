// kda_selective_bwd.hip -- gradients of the selective scan.  With e_t the gradient of h_t,
//     e_t = C_t dy'_t + e^{dt_{t+1} A} e_{t+1},       dy' = dy silu(z)
//     dx_t = dt_t (e_t . B_t) + D dy'_t,              dB_t = sum_c dt_t x_t e_t,  dC_t = sum_c dy'_t h_t
//     d(dt_t) = x_t (e_t . B_t) + A . m_t,            m_t = e^{dt_t A} e_t h_{t-1},  dA = sum_t dt_t m_t
// A wave walks a segment backwards in blocks of K tokens: from the kept state before the block
// it forms the block's states in registers, then goes back over them with e.  A channel is a
// lane (kda_selective.h), so sums over the state's entries stay in a lane, and dB and dC are sums
// over the lanes of a wave; the waves' shares are added by a last launch.
#include "kda_selective.h"

namespace kda {

__device__ __forceinline__ void swap32(float& a, float& b) { asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(a), "+v"(b)); }
__device__ __forceinline__ void swap16(float& a, float& b) { asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(a), "+v"(b)); }

// One halving: lanes with `bit` set take the sums of the upper half of v, the others of the lower;
// CTRL pairs each lane with one whose bit differs.
template <int V, int CTRL> __device__ __forceinline__ void halve(float (&v)[V], int live, int bit) {
    const bool up = threadIdx.x & bit;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        if (i >= live / 2) break;
        const float keep = up ? v[i + live / 2] : v[i], give = up ? v[i] : v[i + live / 2];
        v[i] = keep + dpp<CTRL>(give);
    }
}
// Sums of S values over the 64 lanes: lane l returns the one of value l S / 64.
template <int S> __device__ __forceinline__ float lane_sums(float (&v)[S]) {
#pragma unroll
    for (int i = 0; i < S / 2; ++i) {
        swap32(v[i], v[i + S / 2]);
        v[i] += v[i + S / 2];
    }
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        swap16(v[i], v[i + S / 4]);
        v[i] += v[i + S / 4];
    }
    halve<S, 0x140>(v, S / 4, 8);                 // mirrored in 16 lanes
    if constexpr (S >= 16) halve<S, 0x141>(v, S / 8, 4);   // mirrored in 8
    else v[0] += dpp<0x141>(v[0]);
    if constexpr (S >= 32) halve<S, 0x4e>(v, S / 16, 2);   // lanes 2, 3, 0, 1 of four
    else v[0] += dpp<0x4e>(v[0]);
    return v[0] + dpp<0xb1>(v[0]);                // lanes 1, 0, 3, 2
}

template <typename T, int S>
__global__ __launch_bounds__(kLayerThreads, S == 32 ? 1 : 2) void selective_grads_kernel(SelectiveParams p) {
    constexpr int K = selective_kept(S);
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if (wave >= p.waves) return;
    const Channels ch(p, wave);
    const int lane = threadIdx.x & 63;
    float A2[S], g[S], dA[S], dD = 0.f, dbias = 0.f;
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
    const int64_t state = ((int64_t)s.n * p.C + ch.c) * S, slot = ((int64_t)blockIdx.x * p.C + ch.c) * S;
#pragma unroll
    for (int n = 0; n < S; ++n) { g[n] = 0.f; dA[n] = 0.f; }
    const float* enter = s.j > 0 ? p.seg + slot : p.s0 ? p.s0 + state : nullptr;
    const float* leave = !s.last ? p.rseg + slot : p.dsf ? p.dsf + state : nullptr;
    if (s.begin < s.end || s.last) {
        if (leave) load_entries<S>(g, leave);
        const float bias = p.bias ? p.bias[ch.c] : 0.f, skip = p.D ? p.D[ch.c] : 0.f;
        const T* x = (const T*)p.x + ch.c;
        const T* dt = (const T*)p.dt + ch.c;
        const T* dy = (const T*)p.dy + ch.c;
        const T* z = p.z ? (const T*)p.z + ch.c : dy;
        const int64_t z_stride = p.z ? p.z_stride : p.C;
        const T* B = (const T*)p.B + (int64_t)ch.group * S;
        const T* C = (const T*)p.Cm + (int64_t)ch.group * S;
        const int64_t blocks = (s.end - s.begin + K - 1) / K, first = s.lo / K + s.n + (s.begin - s.lo) / K;
        for (int64_t i = blocks - 1; i >= 0; --i) {
            const int64_t t0 = s.begin + i * K;
            const int count = (int)(s.end - t0 < K ? s.end - t0 : K);
            float h[K + 1][S], d[K];
            T tx[K], td[K], tg[K], tz[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t t = t0 + (k < count ? k : count - 1);
                tx[k] = x[t * p.x_stride];
                td[k] = dt[t * p.dt_stride];
                tg[k] = dy[t * p.C];
                tz[k] = z[t * z_stride];
            }
            if (enter) load_entries<S>(h[0], enter);
            else
#pragma unroll
                for (int n = 0; n < S; ++n) h[0][n] = 0.f;
            if (i > 0) {                          // own state, and what is left of the entering one
                const int64_t at = (first + i) * p.C + ch.c;
                float own[S];
                load_entries<S>(own, p.border + at * S);
                const float sum = p.bdt[at];
#pragma unroll
                for (int n = 0; n < S; ++n) h[0][n] = enter ? __builtin_fmaf(fast_exp2(sum * A2[n]), h[0][n], own[n]) : own[n];
            }
            UniformRow<T, S> nb, nc;
            nb.load(B + t0 * p.b_stride);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (k >= count) break;
                const UniformRow<T, S> b = nb;
                nb.load(B + (t0 + (k + 1 < count ? k + 1 : k)) * p.b_stride);   // the last stays for the way back
                d[k] = step_size(to_f32(td[k]), bias, p.softplus);
                const float w = ch.valid ? d[k] * to_f32(tx[k]) : 0.f;
#pragma unroll
                for (int n = 0; n < S; ++n) h[k + 1][n] = __builtin_fmaf(fast_exp2(d[k] * A2[n]), h[k][n], w * b[n]);
            }
            nc.load(C + (t0 + count - 1) * p.c_stride);
#pragma unroll
            for (int k = K - 1; k >= 0; --k) {
                if (k >= count) continue;
                const int64_t t = t0 + k;
                const UniformRow<T, S> b = nb, c = nc;
                const int64_t ahead = k > 0 ? t - 1 : t;
                nb.load(B + ahead * p.b_stride);
                nc.load(C + ahead * p.c_stride);
                const float xv = to_f32(tx[k]), w = ch.valid ? d[k] * xv : 0.f;
                float dyv = ch.valid ? to_f32(tg[k]) : 0.f;
                if (p.z) {
                    const float zv = to_f32(tz[k]), sig = sigmoid_fast(zv);
                    float y[4] = {skip * xv, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n = 0; n < S; ++n) y[n & 3] = __builtin_fmaf(h[k + 1][n], c[n], y[n & 3]);
                    const float o = (y[0] + y[1]) + (y[2] + y[3]);
                    if (ch.valid) store_out(p.dz, t * p.C + ch.c, dyv * o * sig * __builtin_fmaf(zv, 1.f - sig, 1.f), p.out_bf16);
                    dyv *= zv * sig;
                }
                float v[S], du[4] = {0.f, 0.f, 0.f, 0.f}, dd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int n = 0; n < S; ++n) v[n] = dyv * h[k + 1][n];
                const float dC = lane_sums<S>(v);
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    const float e = __builtin_fmaf(dyv, c[n], g[n]);
                    v[n] = w * e;
                    du[n & 3] = __builtin_fmaf(e, b[n], du[n & 3]);
                    g[n] = fast_exp2(d[k] * A2[n]) * e;
                    const float m = g[n] * h[k][n];
                    dd[n & 3] = __builtin_fmaf(m, A2[n], dd[n & 3]);
                    dA[n] = __builtin_fmaf(m, d[k], dA[n]);
                }
                const float dB = lane_sums<S>(v);
                constexpr int R = 64 / S;         // lanes with the same sum
                if ((lane & (R - 1)) < 2) {
                    float* part = p.bc_part + (t * p.waves + wave) * (2 * S);
                    part[(lane & 1) * S + lane / R] = lane & 1 ? dC : dB;
                }
                const float dus = (du[0] + du[1]) + (du[2] + du[3]);
                float ddt = __builtin_fmaf(dus, xv, ((dd[0] + dd[1]) + (dd[2] + dd[3])) * kLn2);
                if (p.softplus) ddt *= sigmoid_fast(to_f32(td[k]) + bias);
                dD = __builtin_fmaf(dyv, xv, dD);
                dbias += ddt;
                if (ch.valid) {
                    store_out(p.ddt, t * p.C + ch.c, ddt, p.out_bf16);
                    store_out(p.dx, t * p.C + ch.c, __builtin_fmaf(skip, dyv, dus * d[k]), p.out_bf16);
                }
            }
        }
        if (s.j == 0 && p.ds0 && ch.valid) store_entries<S>(p.ds0 + state, g);
    }
    if (!ch.valid) return;
    float* part = p.par_part + (int64_t)blockIdx.x * p.C * (S + 2) + ch.c;
#pragma unroll
    for (int n = 0; n < S; ++n) part[(int64_t)n * p.C] = dA[n];
    part[(int64_t)S * p.C] = dD;
    part[(int64_t)(S + 1) * p.C] = dbias;
}

// dB and dC of a token and group from the shares of its waves.
__global__ __launch_bounds__(kLayerThreads) void selective_bc_kernel(SelectiveParams p, int S) {
    const int64_t i = (int64_t)blockIdx.x * kLayerThreads + threadIdx.x, rows = p.T * p.G;
    const int64_t tg = i / (2 * S);
    if (tg >= rows) return;
    if (p.cu && tg / p.G >= p.cu[p.N]) return;    // rows behind the last document stay as they were
    const int e = (int)(i % (2 * S));
    const float* part = p.bc_part + (tg / p.G * p.waves + tg % p.G * p.group_waves) * (2 * S) + e;
    float sum = 0.f;
#pragma unroll 4
    for (int w = 0; w < p.group_waves; ++w) sum += part[(int64_t)w * 2 * S];
    if (e < S) store_out(p.dB, tg * S + e, sum, p.out_bf16);
    else store_out(p.dC, tg * S + e - S, sum, p.out_bf16);
}

// ---------------------------------------------------------------- launches
template <typename T, int S> static void grads_launch(const SelectiveParams& p, hipStream_t stream) {
    hipLaunchKernelGGL((selective_grads_kernel<T, S>), dim3((unsigned)p.slots, (unsigned)((p.waves + 3) / 4)), dim3(kLayerThreads), 0, stream, p);
}
template <typename T> static void grads_size(const SelectiveParams& p, int S, hipStream_t stream) {
    if (S == 8) grads_launch<T, 8>(p, stream);
    else if (S == 16) grads_launch<T, 16>(p, stream);
    else grads_launch<T, 32>(p, stream);
}
hipError_t launch_selective_grads(const SelectiveParams& p, int S, int in_bf16, hipStream_t stream) {
    if (in_bf16) grads_size<bf16>(p, S, stream);
    else grads_size<float>(p, S, stream);
    const int64_t threads = p.T * p.G * 2 * S;
    if (threads) hipLaunchKernelGGL(selective_bc_kernel, dim3((unsigned)((threads + kLayerThreads - 1) / kLayerThreads)), dim3(kLayerThreads), 0, stream, p, S);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const PartSums sums = {p.par_part, p.slots, S + 2, p.C, S, p.dA, {p.dD, p.dbias}};
    return launch_part_sums(sums, stream);
}

}  // namespace kda
