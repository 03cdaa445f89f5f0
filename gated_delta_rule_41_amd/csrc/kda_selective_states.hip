// kda_selective_states.hip -- states across the segments of a document, forward and in reverse:
// every segment's own sum from a zero state, its share of the gradient of the state that enters
// it, and the carries along the segments.  The own sums walk as the forward does
// (kda_selective.h), without the output's multiply-add: 7 issue slots an entry and token.
#include "kda_selective.h"

namespace kda {

// KEEP 0: own sums of all segments but a document's last.  KEEP > 0: of all, and the own state
// before every KEEP tokens with the sum of dt up to there, for the backward.
template <typename T, int S, int KEEP>
__global__ __launch_bounds__(kLayerThreads) void selective_states_kernel(SelectiveParams p) {
    constexpr int U = KEEP ? KEEP : 4;
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if (s.begin >= s.end || (!KEEP && s.last) || wave >= p.waves) return;
    const Channels ch(p, wave);
    float A2[S], h[S], sum = 0.f;
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
#pragma unroll
    for (int n = 0; n < S; ++n) h[n] = 0.f;
    const float bias = p.bias ? p.bias[ch.c] : 0.f;
    const T* x = (const T*)p.x + ch.c;
    const T* dt = (const T*)p.dt + ch.c;
    const T* B = (const T*)p.B + (int64_t)ch.group * S;
    T nx[U], nd[U];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = t + u < s.end ? t + u : s.end - 1;
            nx[u] = x[at * p.x_stride];
            nd[u] = dt[at * p.dt_stride];
        }
    };
    load(s.begin);
    UniformRow<T, S> nb;
    nb.load(B + s.begin * p.b_stride);
    const int64_t block = KEEP ? s.lo / KEEP + s.n : 0;
    for (int64_t t = s.begin; t < s.end; t += U) {
        T cx[U], cd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) { cx[u] = nx[u]; cd[u] = nd[u]; }
        if (t + U < s.end) load(t + U);
        if constexpr (KEEP != 0) {
            if (t > s.begin && ch.valid) {
                const int64_t at = (block + (t - s.lo) / KEEP) * p.C + ch.c;
                store_entries<S>(p.border + at * S, h);
                p.bdt[at] = sum;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= s.end) break;
            const UniformRow<T, S> b = nb;
            nb.load(B + (t + u + 1 < s.end ? t + u + 1 : s.end - 1) * p.b_stride);
            const float d = step_size(to_f32(cd[u]), bias, p.softplus), w = d * to_f32(cx[u]);
            sum += d;
#pragma unroll
            for (int n = 0; n < S; ++n) h[n] = __builtin_fmaf(fast_exp2(d * A2[n]), h[n], w * b[n]);
        }
    }
    if (!ch.valid) return;
    store_entries<S>(p.seg + ((int64_t)blockIdx.x * p.C + ch.c) * S, h);
    p.sdt[(int64_t)blockIdx.x * p.C + ch.c] = sum;
}

// The gradient of the state that enters a segment, from the segment's own outputs:
//     e_t = C_t dy_t silu(z_t) + e^{dt_{t+1} A} e_{t+1},  e^{dt A} e at its first token.
template <typename T, int S>
__global__ __launch_bounds__(kLayerThreads) void selective_rstates_kernel(SelectiveParams p) {
    constexpr int U = 4;
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if (s.begin >= s.end || s.j == 0 || wave >= p.waves) return;
    const Channels ch(p, wave);
    float A2[S], e[S];
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
#pragma unroll
    for (int n = 0; n < S; ++n) e[n] = 0.f;
    const float bias = p.bias ? p.bias[ch.c] : 0.f;
    const T* dy = (const T*)p.dy + ch.c;
    const T* dt = (const T*)p.dt + ch.c;
    const T* z = p.z ? (const T*)p.z + ch.c : dy;
    const int64_t z_stride = p.z ? p.z_stride : p.C;
    const T* C = (const T*)p.Cm + (int64_t)ch.group * S;
    T ng[U], nd[U], nz[U];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = t - u > s.begin ? t - u : s.begin;
            ng[u] = dy[at * p.C];
            nd[u] = dt[at * p.dt_stride];
            nz[u] = z[at * z_stride];
        }
    };
    load(s.end - 1);
    UniformRow<T, S> nc;
    nc.load(C + (s.end - 1) * p.c_stride);
    for (int64_t t = s.end - 1; t >= s.begin; t -= U) {
        T cg[U], cd[U], cz[U];
#pragma unroll
        for (int u = 0; u < U; ++u) { cg[u] = ng[u]; cd[u] = nd[u]; cz[u] = nz[u]; }
        if (t - U >= s.begin) load(t - U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t - u < s.begin) break;
            const UniformRow<T, S> c = nc;
            nc.load(C + (t - u > s.begin ? t - u - 1 : s.begin) * p.c_stride);
            const float d = step_size(to_f32(cd[u]), bias, p.softplus);
            float g = to_f32(cg[u]);
            if (p.z) {
                const float zv = to_f32(cz[u]);
                g *= zv * sigmoid_fast(zv);
            }
#pragma unroll
            for (int n = 0; n < S; ++n) e[n] = fast_exp2(d * A2[n]) * __builtin_fmaf(g, c[n], e[n]);
        }
    }
    if (ch.valid) store_entries<S>(p.rseg + ((int64_t)blockIdx.x * p.C + ch.c) * S, e);
}

// Along a document's segments, one thread for four entries of a channel: what entered the
// document and the segments' own sums become the states entering the segments (or, from the
// document's end, the gradients of the states leaving them).
struct CarryDir {
    const float* first;       // [N,C,S] or nullptr (zero)
    float* seg;
    bool rev;
};
__global__ __launch_bounds__(kLayerThreads) void selective_carry_kernel(SelectiveParams p, int S) {
    const int64_t i = ((int64_t)blockIdx.y * kLayerThreads + threadIdx.x) * 4, per = (int64_t)p.C * S;
    if (i >= per) return;
    const CarryDir dir = blockIdx.z ? CarryDir{p.dsf, p.rseg, true} : CarryDir{p.s0, p.seg, false};
    const int n = blockIdx.x;
    const int64_t lo = doc_start(p.cu, n, p.seqlen, p.T);
    int64_t hi = doc_start(p.cu, n + 1, p.seqlen, p.T);
    hi = hi < lo ? lo : hi;
    const int64_t count = (hi - lo + p.len - 1) / p.len, slot = lo / p.len + n;
    if (count < 2) return;                        // the walk reads the document's own state
    const f32x4 A2 = *reinterpret_cast<const f32x4*>(p.A + i) * kLog2e;
    f32x4 h = {0.f, 0.f, 0.f, 0.f};
    if (dir.first) h = *reinterpret_cast<const f32x4*>(dir.first + n * per + i);
    constexpr int U = 8;                          // segments on their way
    const int c = (int)(i / S);
    auto at = [&](int64_t j) { return dir.rev ? slot + count - 1 - j : slot + j; };
    for (int64_t j = 0; j + 1 < count; j += U) {
        f32x4 own[U];
        float sum[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = at(j + u + 1 < count ? j + u : count - 2);
            own[u] = *reinterpret_cast<const f32x4*>(dir.seg + k * per + i);
            sum[u] = p.sdt[k * p.C + c];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u + 1 >= count) break;
            *reinterpret_cast<f32x4*>(dir.seg + at(j + u) * per + i) = h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = __builtin_fmaf(fast_exp2(sum[u] * A2[e]), h[e], own[u][e]);
        }
    }
    *reinterpret_cast<f32x4*>(dir.seg + at(count - 1) * per + i) = h;
}

// ---------------------------------------------------------------- launches
template <typename T, int S> static void states_launch(const SelectiveParams& p, bool backward, hipStream_t stream) {
    const dim3 grid((unsigned)p.slots, (unsigned)((p.waves + 3) / 4)), threads(kLayerThreads);
    if (!backward) {
        hipLaunchKernelGGL((selective_states_kernel<T, S, 0>), grid, threads, 0, stream, p);
    } else {
        hipLaunchKernelGGL((selective_states_kernel<T, S, selective_kept(S)>), grid, threads, 0, stream, p);
        if (p.cut) hipLaunchKernelGGL((selective_rstates_kernel<T, S>), grid, threads, 0, stream, p);
    }
    if (!p.cut) return;
    const int64_t pieces = (int64_t)p.C * S / 4;
    hipLaunchKernelGGL(selective_carry_kernel, dim3((unsigned)p.N, (unsigned)((pieces + kLayerThreads - 1) / kLayerThreads), backward ? 2 : 1), threads, 0, stream, p, S);
}
template <typename T> static void states_size(const SelectiveParams& p, int S, bool backward, hipStream_t stream) {
    if (S == 8) states_launch<T, 8>(p, backward, stream);
    else if (S == 16) states_launch<T, 16>(p, backward, stream);
    else states_launch<T, 32>(p, backward, stream);
}
hipError_t launch_selective_states(const SelectiveParams& p, int S, int in_bf16, bool backward, hipStream_t stream) {
    if (in_bf16) states_size<bf16>(p, S, backward, stream);
    else states_size<float>(p, S, backward, stream);
    return hipGetLastError();
}

}  // namespace kda
