// kda_conv.hip -- short causal convolution of every channel over packed documents:
//     pre_t = b + sum_j w_j x_{t-W+1+j},  y_t = act(pre_t),
// its backward and its step for single tokens.  A thread walks a strip of one document's
// tokens with V channels (eight where rows allow 16-byte accesses), the last W - 1 rows in
// registers, so x is read once but for W - 1 rows a strip; the bytes bound it.
#include "kda_layer.h"

namespace kda {

template <typename T, int V> __device__ __forceinline__ void conv_load(float (&v)[V], const T* p) {
    if constexpr (V == 8) load8(v, p);
    else v[0] = to_f32(*p);
}
template <int V> __device__ __forceinline__ void conv_store(void* p, int64_t i, const float (&v)[V], bool as_bf16) {
    if constexpr (V == 8) store8_out(p, i, v, as_bf16);
    else store_out(p, i, v[0], as_bf16);
}
template <int W, int V> struct ConvWeights {
    float w[W][V], b[V];
    __device__ __forceinline__ ConvWeights(const ConvParams& p, int c) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t at = (int64_t)(c + v) * W;
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = p.weight_bf16 ? to_f32(((const bf16*)p.weight)[at + j]) : ((const float*)p.weight)[at + j];
            b[v] = !p.bias ? 0.f : p.weight_bf16 ? to_f32(((const bf16*)p.bias)[c + v]) : ((const float*)p.bias)[c + v];
        }
    }
};

// Rows t - W + 1 .. t - 1 before token t of document n, oldest first.
template <typename T, int W, int V>
__device__ __forceinline__ void conv_history(float (&h)[W - 1][V], const ConvParams& p, const Segment& s, int64_t t, int c) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int64_t at = t - (W - 1) + r;
        if (at >= s.lo) conv_load<T, V>(h[r], (const T*)p.x + at * p.x_stride + c);
        else if (p.s0) conv_load<T, V>(h[r], (const T*)p.s0 + ((int64_t)s.n * (W - 1) + (W - 1) + (at - s.lo)) * p.C + c);
        else
#pragma unroll
            for (int v = 0; v < V; ++v) h[r][v] = 0.f;
    }
}
template <int W, int V> __device__ __forceinline__ void conv_shift(float (&h)[W - 1][V], const float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int r = 0; r + 1 < W - 1; ++r) h[r][v] = h[r + 1][v];
        h[W - 2][v] = x[v];
    }
}
template <int W, int V>
__device__ __forceinline__ float conv_pre(const ConvWeights<W, V>& k, const float (&h)[W - 1][V], float x, int v) {
    float y = k.b[v];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) y = __builtin_fmaf(k.w[j][v], h[j][v], y);
    return __builtin_fmaf(k.w[W - 1][v], x, y);
}

template <typename T, int W, int V>
__global__ __launch_bounds__(kLayerThreads) void conv_fwd_kernel(ConvParams p) {
    constexpr int U = 4;                          // rows on their way
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int c = (int)(blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= p.C || (s.begin >= s.end && !s.last)) return;
    const ConvWeights<W, V> k(p, c);
    float h[W - 1][V];
    conv_history<T, W, V>(h, p, s, s.begin, c);
    const T* x = (const T*)p.x + c;
    float next[U][V];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < U; ++u) conv_load<T, V>(next[u], x + (t + u < s.end ? t + u : s.end - 1) * p.x_stride);
    };
    if (s.begin < s.end) load(s.begin);
    for (int64_t t = s.begin; t < s.end; t += U) {
        float now[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) now[u][v] = next[u][v];
        if (t + U < s.end) load(t + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= s.end) break;
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                y[v] = conv_pre<W, V>(k, h, now[u][v], v);
                if (p.silu) y[v] *= sigmoid_fast(y[v]);
            }
            conv_shift<W, V>(h, now[u]);
            conv_store<V>(p.y, (t + u) * p.C + c, y, p.out_bf16);
        }
    }
    if (s.last && p.sfinal)
#pragma unroll
        for (int r = 0; r < W - 1; ++r) conv_store<V>(p.sfinal, ((int64_t)s.n * (W - 1) + r) * p.C + c, h[r], sizeof(T) == 2);
}

// dx_s = sum_j w_j dpre_{s+W-1-j} is complete W - 1 tokens later, so a strip goes on for
// W - 1 tokens of its document (dpre = 0 behind it).  The first strip of a document also ends
// the rows of its initial state, in front of it.
template <typename T, int W, int V>
__global__ __launch_bounds__(kLayerThreads) void conv_bwd_kernel(ConvParams p) {
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int c = (int)(blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (c >= p.C) return;
    float dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    if (s.begin < s.end || s.last) {
        const ConvWeights<W, V> k(p, c);
        float h[W - 1][V], d[W][V];               // rows before t; dpre of t - W + 1 .. t
        conv_history<T, W, V>(h, p, s, s.begin, c);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) d[j][v] = 0.f;
        const T* x = (const T*)p.x + c;
        const T* dy = (const T*)p.dy + c;
        float nx[V], ng[V];
        auto load = [&](int64_t t) {
            if (t < s.hi) {
                conv_load<T, V>(nx, x + t * p.x_stride);
                conv_load<T, V>(ng, dy + t * p.C);
            }
        };
        load(s.begin);
        for (int64_t t = s.begin; t < s.end + W - 1; ++t) {
            float g[V], xt[V];
#pragma unroll
            for (int v = 0; v < V; ++v) { xt[v] = nx[v]; g[v] = ng[v]; }
            load(t + 1);
#pragma unroll
            for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) d[j][v] = d[j + 1][v];
            if (t < s.hi) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float f = g[v];
                    if (p.silu) {
                        const float pre = conv_pre<W, V>(k, h, xt[v], v), sig = sigmoid_fast(pre);
                        f *= sig * __builtin_fmaf(pre, 1.f - sig, 1.f);
                    }
                    d[W - 1][v] = f;
                    if (t < s.end) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][v] = __builtin_fmaf(f, h[j][v], dw[j][v]);
                        dw[W - 1][v] = __builtin_fmaf(f, xt[v], dw[W - 1][v]);
                        dw[W][v] += f;
                    }
                }
                conv_shift<W, V>(h, xt);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) d[W - 1][v] = 0.f;
            }
            const int64_t at = t - (W - 1);       // the row that is complete
            if (at < s.begin && (s.j > 0 || !p.ds0)) continue;
            float dx[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dx[v] = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j) dx[v] = __builtin_fmaf(k.w[j][v], d[W - 1 - j][v], dx[v]);
            }
            const int64_t r = at - s.hi + (W - 1);   // its row in the final state
            if (r >= 0 && p.dsf) {
                float e[V];
                conv_load<T, V>(e, (const T*)p.dsf + ((int64_t)s.n * (W - 1) + r) * p.C + c);
#pragma unroll
                for (int v = 0; v < V; ++v) dx[v] += e[v];
            }
            if (at >= s.begin) conv_store<V>(p.dx, at * p.C + c, dx, p.out_bf16);
            else conv_store<V>(p.ds0, ((int64_t)s.n * (W - 1) + (at - s.lo) + (W - 1)) * p.C + c, dx, sizeof(T) == 2);
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j) conv_store<V>(p.part, ((int64_t)blockIdx.x * (W + 1) + j) * p.C + c, dw[j], false);
}

template <typename T, int W, int V>
__global__ __launch_bounds__(kLayerThreads) void conv_decode_kernel(ConvParams p) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, per = p.C / V;
    const int64_t n = i / per;
    const int c = (int)(i % per) * V;
    if (n >= p.N) return;
    float h[W - 1][V], x[V], y[V];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        if (p.s0) conv_load<T, V>(h[r], (const T*)p.s0 + (n * (W - 1) + r) * p.C + c);
        else
#pragma unroll
            for (int v = 0; v < V; ++v) h[r][v] = 0.f;
    }
    conv_load<T, V>(x, (const T*)p.x + n * p.x_stride + c);
    const ConvWeights<W, V> k(p, c);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        y[v] = conv_pre<W, V>(k, h, x[v], v);
        if (p.silu) y[v] *= sigmoid_fast(y[v]);
    }
    conv_shift<W, V>(h, x);
    conv_store<V>(p.y, n * p.C + c, y, p.out_bf16);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) conv_store<V>(p.sfinal, (n * (W - 1) + r) * p.C + c, h[r], sizeof(T) == 2);
}

// ---------------------------------------------------------------- launches
enum ConvCall { kConvFwd, kConvBwd, kConvDecode };
template <typename T, int W, int V> static void conv_launch(const ConvParams& p, ConvCall call, hipStream_t stream) {
    const int64_t per = p.C / V;
    if (call == kConvDecode) {
        const int64_t threads = p.N * per;
        hipLaunchKernelGGL((conv_decode_kernel<T, W, V>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, p);
        return;
    }
    const int threads = per >= kLayerThreads ? kLayerThreads : (int)((per + 63) / 64 * 64);
    const dim3 grid((unsigned)p.slots, (unsigned)((per + threads - 1) / threads));
    if (call == kConvFwd) hipLaunchKernelGGL((conv_fwd_kernel<T, W, V>), grid, dim3(threads), 0, stream, p);
    else hipLaunchKernelGGL((conv_bwd_kernel<T, W, V>), grid, dim3(threads), 0, stream, p);
}
template <typename T, int W> static void conv_vec(const ConvParams& p, ConvCall call, hipStream_t stream) {
    if (p.C % 8 == 0 && p.x_stride % 8 == 0) conv_launch<T, W, 8>(p, call, stream);
    else conv_launch<T, W, 1>(p, call, stream);
}
template <typename T> static void conv_width(const ConvParams& p, int W, ConvCall call, hipStream_t stream) {
    if (W == 2) conv_vec<T, 2>(p, call, stream);
    else if (W == 3) conv_vec<T, 3>(p, call, stream);
    else conv_vec<T, 4>(p, call, stream);
}
static hipError_t conv_any(const ConvParams& p, int W, int in_bf16, ConvCall call, hipStream_t stream) {
    if (in_bf16) conv_width<bf16>(p, W, call, stream);
    else conv_width<float>(p, W, call, stream);
    return hipGetLastError();
}
hipError_t launch_conv_fwd(const ConvParams& p, int W, int in_bf16, hipStream_t stream) { return conv_any(p, W, in_bf16, kConvFwd, stream); }
hipError_t launch_conv_decode(const ConvParams& p, int W, int in_bf16, hipStream_t stream) { return conv_any(p, W, in_bf16, kConvDecode, stream); }
hipError_t launch_conv_bwd(const ConvParams& p, int W, int in_bf16, float* dw, float* db, hipStream_t stream) {
    const hipError_t e = conv_any(p, W, in_bf16, kConvBwd, stream);
    if (e != hipSuccess) return e;
    const PartSums s = {p.part, p.slots, W + 1, p.C, W, dw, {db, nullptr}};
    return launch_part_sums(s, stream);
}

}  // namespace kda
