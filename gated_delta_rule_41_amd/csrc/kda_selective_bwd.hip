// kda_selective_bwd.hip -- gradients of the selective scan.  With e_t the gradient of h_t,
//     e_t = C_t dy'_t + e^{dt_{t+1} A} e_{t+1},       dy' = dy silu(z)
//     dx_t = dt_t (e_t . B_t) + D dy'_t,              dB_t = sum_c dt_t x_t e_t,  dC_t = sum_c dy'_t h_t
//     d(dt_t) = x_t (e_t . B_t) + A . m_t,            m_t = e^{dt_t A} e_t h_{t-1},  dA = sum_t dt_t m_t
// A wave walks a segment backwards in blocks of K tokens: from the kept state before the block
// it forms the block's states in registers, then goes back over them with e.  A channel is a
// lane (kda_selective.h), so sums over the state's entries stay in a lane, and dB and dC are sums
// over the lanes of a wave; the waves' shares are added by a last launch.  An entry and token
// costs 15 multiplies and multiply-adds, two exponentials and its share of 70 exchanges and
// additions: vector instructions bound the kernel, which takes 924 us for 4 x 4096 tokens x 4096
// channels of 16 entries (bf16, gated), where the 394 a token (counted) take 672 at one every
// four cycles and 742 with a second slot for the 41 exponentials and quotients among them.
#include "kda_selective.h"

namespace kda {

// Exchanges the upper 32 lanes of a[i] with the lower of b[i] (or odd rows of 16 with even ones), for two pairs; the wait
// is for the values' own instructions.
__device__ __forceinline__ void swap32(float& a0, float& b0, float& a1, float& b1) {
    asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1\n\tv_permlane32_swap_b32 %2, %3" : "+v"(a0), "+v"(b0), "+v"(a1), "+v"(b1));
}
__device__ __forceinline__ void swap16(float& a0, float& b0, float& a1, float& b1) {
    asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1\n\tv_permlane16_swap_b32 %2, %3" : "+v"(a0), "+v"(b0), "+v"(a1), "+v"(b1));
}

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
    for (int i = 0; i < S / 2; i += 2) {
        swap32(v[i], v[i + S / 2], v[i + 1], v[i + 1 + S / 2]);
        v[i] += v[i + S / 2];
        v[i + 1] += v[i + 1 + S / 2];
    }
#pragma unroll
    for (int i = 0; i < S / 4; i += 2) {
        swap16(v[i], v[i + S / 4], v[i + 1], v[i + 1 + S / 4]);
        v[i] += v[i + S / 4];
        v[i + 1] += v[i + 1 + S / 4];
    }
    halve<S, 0x140>(v, S / 4, 8);                 // mirrored in 16 lanes
    if constexpr (S >= 16) halve<S, 0x141>(v, S / 8, 4);   // mirrored in 8
    else v[0] += dpp<0x141>(v[0]);
    if constexpr (S >= 32) halve<S, 0x4e>(v, S / 16, 2);   // lanes 2, 3, 0, 1 of four
    else v[0] += dpp<0x4e>(v[0]);
    return v[0] + dpp<0xb1>(v[0]);                // lanes 1, 0, 3, 2
}

// The kernel's parameters, read again where they are used: held in scalar registers from the start, they would push
// out others.
typedef const __attribute__((address_space(4))) SelectiveParams* ParamsAgain;
__device__ __forceinline__ ParamsAgain params_again() {
    ParamsAgain q = (ParamsAgain)__builtin_amdgcn_kernarg_segment_ptr();
    asm("" : "+s"(q));
    return q;
}

template <typename T, int S, bool GATED>
__global__ __launch_bounds__(kLayerThreads, S == 32 ? 1 : 2) void selective_grads_kernel(SelectiveParams p) {
    constexpr int K = selective_kept(S);
    __shared__ f32x4 enters[4 * (S / 4) * 64];    // the states that enter the waves' segments
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if (wave >= p.waves) return;
    const Channels ch(p, wave);
    const int lane = threadIdx.x & 63;
    constexpr int R = 64 / S;                     // lanes with the same sum over lanes: the first stores dB's, the second dC's
    unsigned part_at = ((lane & 1) * S + lane / R) * 4;
    asm("" : "+v"(part_at));
    float A2[S], g[S], dA[S], dD = 0.f, dbias = 0.f;
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
    const int64_t state = ((int64_t)s.n * p.C + ch.c) * S;
#pragma unroll
    for (int n = 0; n < S; ++n) { g[n] = 0.f; dA[n] = 0.f; }
    if (s.begin < s.end || s.last) {
        if (!s.last) load_kept<S>(g, p.rseg, blockIdx.x, p.C, ch.c);
        else if (p.dsf) load_entries<S>(g, p.dsf + state);
        const float bias = p.bias ? p.bias[ch.c] : 0.f, skip = p.D ? p.D[ch.c] : 0.f;
        // What a block's forward walk begins with, asked for while the block before it is on its way back and
        // most of that one's states are no longer needed.  Nothing is kept before a segment's first block.
        T nx[K], nd[K];
        float own[S], own_dt;
        auto ahead = [&](const int64_t t0, const int count) {
            const ParamsAgain q = params_again();
            const T* x = (const T*)q->x + t0 * q->x_stride;
            const T* dt = (const T*)q->dt + t0 * q->dt_stride;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                nx[k] = row_at(x, ch);
                nd[k] = row_at(dt, ch);
                if (k + 1 < count) { x += q->x_stride; dt += q->dt_stride; }
            }
            const int64_t at = s.lo / K + s.n + (t0 - s.lo) / K;
            load_kept<S>(own, q->border, at, q->C, ch.c);
            own_dt = row_at(q->bdt + at * q->C, ch);
        };
        f32x4* const enter = enters + (threadIdx.x >> 6) * (S / 4) * 64 + lane;
        // the block of `count` tokens from t0 on
        auto block = [&](auto whole, const int64_t t0, const int count) {
            float h[K + 1][S], d[K];
            T tx[K], td[K], tg[K], tz[K];
            {
                const ParamsAgain q = params_again();
                const T* dy = (const T*)q->dy + t0 * q->C;
                const T* z = GATED ? (const T*)q->z + t0 * q->z_stride : dy;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    tx[k] = nx[k];
                    td[k] = nd[k];
                    tg[k] = row_at(dy, ch);
                    if (GATED) tz[k] = row_at(z, ch);
                    if (whole.value || k + 1 < count) { dy += q->C; z += GATED ? q->z_stride : 0; }
                }
            }
            const bool kept = t0 > s.begin;       // own state, and what is left of the entering one
#pragma unroll
            for (int n = 0; n < S; ++n) {
                const float e = enter[n / 4 * 64][n & 3];
                h[0][n] = kept ? __builtin_fmaf(fast_exp2(own_dt * A2[n]), e, own[n]) : e;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                d[k] = step_size(to_f32(td[k]), bias, p.softplus);
            }
            UniformRows<T, S> B((const T*)p.B + t0 * p.b_stride + (int64_t)ch.group * S, p.b_stride);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                __builtin_amdgcn_sched_barrier(0);
                if (!whole.value && k >= count) continue;
                const UniformRow<T, S> b = B.next(whole.value ? k + 1 < K : k + 1 < count);
                const float w = ch.valid ? d[k] * to_f32(tx[k]) : 0.f;
#pragma unroll
                for (int n = 0; n < S; ++n) h[k + 1][n] = __builtin_fmaf(fast_exp2(d[k] * A2[n]), h[k][n], w * b[n]);
            }
            B.step = -p.b_stride;                 // it stands at the block's last token
            asm("" : "+s"(B.p));                  // rows are loaded again, not kept from above
            int64_t t = t0 + count - 1;
            const ParamsAgain r = params_again();
            UniformRows<T, S> C((const T*)r->Cm + t * r->c_stride + (int64_t)ch.group * S, -r->c_stride);
#pragma unroll
            for (int k = K - 1; k >= 0; --k) {
                __builtin_amdgcn_sched_barrier(0);    // or rows of many tokens are loaded at once and spill
                if (!whole.value && k >= count) {
                    if (k == 1) ahead(kept ? t0 - K : t0, kept ? K : count);
                    continue;
                }
                const UniformRow<T, S> b = B.next(k > 0), c = C.next(k > 0);
                float dk = d[k];
                asm("" : "+v"(dk));               // the decays are formed again: kept from above they would take S registers a token
                const float xv = to_f32(tx[k]), w = ch.valid ? dk * xv : 0.f;
                float dyv = ch.valid ? to_f32(tg[k]) : 0.f, dz = 0.f;
                if constexpr (GATED) {
                    const float zv = to_f32(tz[k]), sig = sigmoid_fast(zv);
                    float y[4] = {skip * xv, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n = 0; n < S; ++n) y[n & 3] = __builtin_fmaf(h[k + 1][n], c[n], y[n & 3]);
                    dz = dyv * ((y[0] + y[1]) + (y[2] + y[3])) * sig * __builtin_fmaf(zv, 1.f - sig, 1.f);
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
                    g[n] = fast_exp2(dk * A2[n]) * e;
                    const float m = g[n] * h[k][n];
                    dd[n & 3] = __builtin_fmaf(m, A2[n], dd[n & 3]);
                    dA[n] = __builtin_fmaf(m, dk, dA[n]);
                }
                const float dB = lane_sums<S>(v);
                const float dus = (du[0] + du[1]) + (du[2] + du[3]);
                float ddt = __builtin_fmaf(dus, xv, ((dd[0] + dd[1]) + (dd[2] + dd[3])) * kLn2);
                if (r->softplus) ddt *= sigmoid_fast(to_f32(td[k]) + bias);
                const float dx = __builtin_fmaf(skip, dyv, dus * dk);
                dD = __builtin_fmaf(dyv, xv, dD);
                if (k == 1) ahead(kept ? t0 - K : t0, kept ? K : count);
                dbias += ddt;
                float* part = r->bc_part + (t * r->waves + wave) * (2 * S);
                if ((lane & (R - 1)) < 2) *lane_bytes(part, part_at) = lane & 1 ? dC : dB;
                if (ch.valid) {
                    const int64_t out = t * r->C;
                    if (r->out_bf16) {
                        *lane_of((bf16*)r->dx + out, ch) = (bf16)dx;
                        *lane_of((bf16*)r->ddt + out, ch) = (bf16)ddt;
                        if (GATED) *lane_of((bf16*)r->dz + out, ch) = (bf16)dz;
                    } else {
                        *lane_of((float*)r->dx + out, ch) = dx;
                        *lane_of((float*)r->ddt + out, ch) = ddt;
                        if (GATED) *lane_of((float*)r->dz + out, ch) = dz;
                    }
                }
                --t;
            }
        };
        {
            float e[S];
            if (s.j > 0) load_kept<S>(e, p.seg, blockIdx.x, p.C, ch.c);
            else if (p.s0) load_entries<S>(e, p.s0 + state);
            else
#pragma unroll
                for (int n = 0; n < S; ++n) e[n] = 0.f;
#pragma unroll
            for (int n = 0; n < S; n += 4) enter[n / 4 * 64] = f32x4{e[n], e[n + 1], e[n + 2], e[n + 3]};   // a wave's own
        }
        int64_t t0 = s.begin + (s.end - s.begin) / K * K;
        if (t0 < s.end) ahead(t0, (int)(s.end - t0));
        else if (s.begin < s.end) ahead(t0 - K, K);
        if (t0 < s.end) block(std::false_type(), t0, (int)(s.end - t0));
        for (t0 -= K; t0 >= s.begin; t0 -= K) block(std::true_type(), t0, K);
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
    const dim3 grid((unsigned)p.slots, (unsigned)((p.waves + 3) / 4));
    if (p.z) hipLaunchKernelGGL((selective_grads_kernel<T, S, true>), grid, dim3(kLayerThreads), 0, stream, p);
    else hipLaunchKernelGGL((selective_grads_kernel<T, S, false>), grid, dim3(kLayerThreads), 0, stream, p);
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
