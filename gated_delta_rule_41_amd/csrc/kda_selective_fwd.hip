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
    constexpr int U = 4;                          // tokens a block: their loads are one block ahead
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if ((s.begin >= s.end && !s.last) || wave >= p.waves) return;
    const Channels ch(p, wave);
    float A2[S], h[S];
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
    const int64_t state = ((int64_t)s.n * p.C + ch.c) * S;
    if (s.j > 0) load_kept<S>(h, p.seg, blockIdx.x, p.C, ch.c);
    else if (p.s0) load_entries<S>(h, p.s0 + state);
    else
#pragma unroll
        for (int n = 0; n < S; ++n) h[n] = 0.f;
    if (s.begin < s.end) {
        const float bias = p.bias ? p.bias[ch.c] : 0.f, skip = p.D ? p.D[ch.c] : 0.f;
        const T* x = (const T*)p.x + s.begin * p.x_stride;
        const T* dt = (const T*)p.dt + s.begin * p.dt_stride;
        const int64_t z_stride = p.z ? p.z_stride : p.x_stride;
        const T* z = p.z ? (const T*)p.z + s.begin * z_stride : x;
        UniformRows<T, S> B((const T*)p.B + s.begin * p.b_stride + (int64_t)ch.group * S, p.b_stride);
        UniformRows<T, S> C((const T*)p.Cm + s.begin * p.c_stride + (int64_t)ch.group * S, p.c_stride);
        int64_t out = s.begin * p.C;
        T nx[U], nd[U], nz[U];
        int left = (int)(s.end - s.begin);        // tokens from the block on
        auto load = [&](int count) {              // the block at x, dt, z; rows behind the segment are its last
#pragma unroll
            for (int u = 0; u < U; ++u) {
                nx[u] = row_at(x, ch);
                nd[u] = row_at(dt, ch);
                nz[u] = row_at(z, ch);
                if (u + 1 < count) { x += p.x_stride; dt += p.dt_stride; z += z_stride; }
            }
        };
        load(left);
        auto block = [&](auto whole, int count) {
            float d[U], w[U], o[U];
            T cx[U], cz[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                d[u] = step_size(to_f32(nd[u]), bias, p.softplus);
                w[u] = d[u] * to_f32(nx[u]);
                cx[u] = nx[u];
                cz[u] = nz[u];
            }
            if (whole.value ? left > U : false) load(left - U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!whole.value && u >= count) break;
                const UniformRow<T, S> b = B.next(u + 1 < left), c = C.next(u + 1 < left);
                float y[4] = {skip * to_f32(cx[u]), 0.f, 0.f, 0.f};   // four sums, so that they need not wait for one another
#pragma unroll
                for (int n = 0; n < S; ++n) {
                    h[n] = __builtin_fmaf(fast_exp2(d[u] * A2[n]), h[n], w[u] * b[n]);
                    y[n & 3] = __builtin_fmaf(h[n], c[n], y[n & 3]);
                }
                o[u] = (y[0] + y[1]) + (y[2] + y[3]);
            }
            if (p.z)
#pragma unroll
                for (int u = 0; u < U; ++u) o[u] *= to_f32(cz[u]) * sigmoid_fast(to_f32(cz[u]));
            if (ch.valid)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (whole.value || u < count) row_put(p.y, out + (int64_t)u * p.C, ch, o[u], p.out_bf16);
        };
        for (; left >= U; left -= U, out += (int64_t)U * p.C) block(std::true_type(), U);
        if (left > 0) block(std::false_type(), left);
    }
    if (s.last && p.sfinal && ch.valid) store_entries<S>(p.sfinal + state, h);
}

// One token of every sequence: S / 4 lanes share a channel with four entries each, so that the
// state moves in 16-byte pieces side by side; it is read and written once, which bounds the step:
// 256 sequences x 4096 channels of 16 entries take 30 us, 4.8 TB/s.
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
