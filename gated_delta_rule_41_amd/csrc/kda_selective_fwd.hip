// kda_selective_fwd.hip -- the selective scan forward over packed documents:
//     h_t = e^{dt_t A} h_{t-1} + dt_t x_t B_t,  y_t = (C_t . h_t + D x_t) silu(z_t).
// A wave walks one segment of a document with 64 channels (kda_selective.h).  Documents longer
// than a segment are walked twice: first every segment from a zero state, which leaves its own
// sum and the sum of its dt, then a carry along the segments (h <- e^{A sum dt} h + own), then
// every segment again from the state that enters it.
#include "kda_selective.h"

namespace kda {

template <typename T, int S>
__global__ __launch_bounds__(kLayerThreads) void selective_out_kernel(SelectiveParams p) {
    constexpr int U = 4;
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if ((s.begin >= s.end && !s.last) || wave >= p.waves) return;
    const Channels ch(p, wave);
    float A2[S], h[S];
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
    const int64_t state = ((int64_t)s.n * p.C + ch.c) * S;
    if (s.j > 0) load_entries<S>(h, p.seg + ((int64_t)blockIdx.x * p.C + ch.c) * S);
    else if (p.s0) load_entries<S>(h, p.s0 + state);
    else
#pragma unroll
        for (int n = 0; n < S; ++n) h[n] = 0.f;
    if (s.begin < s.end) {
        const float bias = p.bias ? p.bias[ch.c] : 0.f, skip = p.D ? p.D[ch.c] : 0.f;
        const T* x = (const T*)p.x + ch.c;
        const T* dt = (const T*)p.dt + ch.c;
        const T* z = p.z ? (const T*)p.z + ch.c : x;
        const int64_t z_stride = p.z ? p.z_stride : p.x_stride;
        const T* B = (const T*)p.B + (int64_t)ch.group * S;
        const T* C = (const T*)p.Cm + (int64_t)ch.group * S;
        T nx[U], nd[U], nz[U];
        auto load = [&](int64_t t) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = t + u < s.end ? t + u : s.end - 1;
                nx[u] = x[at * p.x_stride];
                nd[u] = dt[at * p.dt_stride];
                nz[u] = z[at * z_stride];
            }
        };
        load(s.begin);
        UniformRow<T, S> nb, nc;
        nb.load(B + s.begin * p.b_stride);
        nc.load(C + s.begin * p.c_stride);
        for (int64_t t = s.begin; t < s.end; t += U) {
            T cx[U], cd[U], cz[U];
#pragma unroll
            for (int u = 0; u < U; ++u) { cx[u] = nx[u]; cd[u] = nd[u]; cz[u] = nz[u]; }
            if (t + U < s.end) load(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= s.end) break;
                const UniformRow<T, S> b = nb, c = nc;
                const int64_t at = t + u + 1 < s.end ? t + u + 1 : s.end - 1;
                nb.load(B + at * p.b_stride);
                nc.load(C + at * p.c_stride);
                const float d = step_size(to_f32(cd[u]), bias, p.softplus), xv = to_f32(cx[u]), w = d * xv;
                float y[4] = {skip * xv, 0.f, 0.f, 0.f};      // four sums, so that they need not wait for one another
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    h[n] = __builtin_fmaf(fast_exp2(d * A2[n]), h[n], w * b[n]);
                    y[n & 3] = __builtin_fmaf(h[n], c[n], y[n & 3]);
                }
                float o = (y[0] + y[1]) + (y[2] + y[3]);
                if (p.z) {
                    const float zv = to_f32(cz[u]);
                    o *= zv * sigmoid_fast(zv);
                }
                if (ch.valid) store_out(p.y, (t + u) * p.C + ch.c, o, p.out_bf16);
            }
        }
    }
    if (s.last && p.sfinal && ch.valid) store_entries<S>(p.sfinal + state, h);
}

// One token of every sequence: S / 4 lanes share a channel with four entries each, so that the
// state moves in 16-byte pieces side by side; it is read and written once, which bounds the step.
template <typename T, int S>
__global__ __launch_bounds__(kLayerThreads) void selective_decode_kernel(SelectiveParams p) {
    constexpr int L = S / 4;
    const int64_t i = (int64_t)blockIdx.x * kLayerThreads + threadIdx.x, nc = i / L;
    const int e = (int)(i % L) * 4;
    if (nc >= (int64_t)p.N * p.C) return;         // whole channels: S / 4 lanes are next to each other
    const int64_t n = nc / p.C;
    const int c = (int)(nc % p.C), g = c / (p.C / p.G);
    f32x4 h = {0.f, 0.f, 0.f, 0.f};
    if (p.s0) h = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p.s0 + nc * S + e));
    const f32x4 A = *reinterpret_cast<const f32x4*>(p.A + (int64_t)c * S + e) * kLog2e;
    const f32x4 b = unpack4(*reinterpret_cast<const typename V4<T>::t*>((const T*)p.B + n * p.b_stride + (int64_t)g * S + e));
    const f32x4 cm = unpack4(*reinterpret_cast<const typename V4<T>::t*>((const T*)p.Cm + n * p.c_stride + (int64_t)g * S + e));
    const float x = to_f32(((const T*)p.x)[n * p.x_stride + c]);
    const float d = step_size(to_f32(((const T*)p.dt)[n * p.dt_stride + c]), p.bias ? p.bias[c] : 0.f, p.softplus), w = d * x;
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = __builtin_fmaf(fast_exp2(d * A[j]), h[j], w * b[j]);
        y = __builtin_fmaf(h[j], cm[j], y);
    }
    __builtin_nontemporal_store(h, reinterpret_cast<f32x4*>(p.sfinal + nc * S + e));
#pragma unroll
    for (int m = 1; m < L; m <<= 1) y += __shfl_xor(y, m, 64);
    if (e) return;
    if (p.D) y = __builtin_fmaf(p.D[c], x, y);
    if (p.z) {
        const float z = to_f32(((const T*)p.z)[n * p.z_stride + c]);
        y *= z * sigmoid_fast(z);
    }
    store_out(p.y, nc, y, p.out_bf16);
}

// ---------------------------------------------------------------- launches
enum SelectiveCall { kOut, kDecode };
template <typename T, int S> static void selective_launch(const SelectiveParams& p, SelectiveCall call, hipStream_t stream) {
    if (call == kDecode) {
        const int64_t threads = (int64_t)p.N * p.C * (S / 4);
        hipLaunchKernelGGL((selective_decode_kernel<T, S>), dim3((unsigned)((threads + kLayerThreads - 1) / kLayerThreads)), dim3(kLayerThreads), 0, stream, p);
        return;
    }
    const dim3 grid((unsigned)p.slots, (unsigned)((p.waves + 3) / 4));
    hipLaunchKernelGGL((selective_out_kernel<T, S>), grid, dim3(kLayerThreads), 0, stream, p);
}
template <typename T> static void selective_size(const SelectiveParams& p, int S, SelectiveCall call, hipStream_t stream) {
    if (S == 8) selective_launch<T, 8>(p, call, stream);
    else if (S == 16) selective_launch<T, 16>(p, call, stream);
    else selective_launch<T, 32>(p, call, stream);
}
static hipError_t selective_any(const SelectiveParams& p, int S, int in_bf16, SelectiveCall call, hipStream_t stream) {
    if (in_bf16) selective_size<bf16>(p, S, call, stream);
    else selective_size<float>(p, S, call, stream);
    return hipGetLastError();
}
hipError_t launch_selective_out(const SelectiveParams& p, int S, int in_bf16, hipStream_t stream) { return selective_any(p, S, in_bf16, kOut, stream); }
hipError_t launch_selective_decode(const SelectiveParams& p, int S, int in_bf16, hipStream_t stream) { return selective_any(p, S, in_bf16, kDecode, stream); }

}  // namespace kda
