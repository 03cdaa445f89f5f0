// kda_conv.hip -- short causal convolution of every channel over packed documents:
//     pre_t = b + sum_j w_j x_{t-W+1+j},  y_t = act(pre_t),
// its backward and its step for single tokens.  A thread walks a strip of one document's
// tokens with V channels (eight or one), the last W - 1 rows in registers, so x is read once but
// for W - 1 rows a strip; the bytes bound it: bf16, 4 taps, 16411 x 12288 forward 157 us (5.2
// TB/s), 32768 x 4096 backward 162 (5.0), a step of 256 x 12288 9.8 (5.1).
#include "kda_layer.h"

namespace kda {

// A row's V channels as they lie in memory.
template <typename T, int V> struct ConvRow : Raw8<T> {};
template <typename T> struct ConvRow<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T* p) { r = *p; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f32(r); }
};
template <typename T, int V> __device__ __forceinline__ void conv_load(float (&v)[V], const T* p) {
    ConvRow<T, V> r;
    r.load(p);
    r.get(v);
}
template <int V, bool STREAM = false> __device__ __forceinline__ void conv_store(void* p, int64_t i, const float (&v)[V], bool as_bf16) {
    if constexpr (V == 8) store8_out<STREAM>(p, i, v, as_bf16);
    else store_out(p, i, v[0], as_bf16);
}
// A thread's first channel.  The last of a row's threads moves back where channels are left over, and does some of its
// neighbour's again: both write the same values.
template <int V> __device__ __forceinline__ int conv_channel(int64_t thread, int C) {
    const int64_t c = thread * V;
    return (int)(c + V <= C ? c : C - V);
}

template <int W, int V> struct ConvWeights {
    float w[W][V], b[V];
    template <typename T> __device__ __forceinline__ void load(const T* weight, const T* bias, int c) {
        const T* p = weight + (int64_t)c * W;
#pragma unroll
        for (int v = 0; v < V; ++v) b[v] = 0.f;
        if constexpr (V > 1) {                    // V channels' taps lie side by side: W pieces of V
            float part[W][V];
#pragma unroll
            for (int i = 0; i < W; ++i) conv_load<T, V>(part[i], p + V * i);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < W; ++j) w[j][v] = part[(v * W + j) / V][(v * W + j) % V];
            if (bias) conv_load<T, V>(b, bias + c);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][0] = to_f32(p[j]);
            if (bias) b[0] = to_f32(bias[c]);
        }
    }
    __device__ __forceinline__ ConvWeights(const ConvParams& p, int c) {
        if (p.weight_bf16) load((const bf16*)p.weight, (const bf16*)p.bias, c);
        else load((const float*)p.weight, (const float*)p.bias, c);
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
    const int64_t thread = blockIdx.y * blockDim.x + threadIdx.x;
    const int c = conv_channel<V>(thread, p.C);
    if (thread * V >= p.C || (s.begin >= s.end && !s.last)) return;
    const ConvWeights<W, V> k(p, c);
    float h[W - 1][V];
    conv_history<T, W, V>(h, p, s, s.begin, c);
    const T* x = (const T*)p.x + s.begin * p.x_stride + c;
    ConvRow<T, V> next[U];
    int left = (int)(s.end - s.begin);            // tokens from the block on
    auto load = [&](int count) {                  // rows behind the strip are its last
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next[u].load(x);
            if (u + 1 < count) x += p.x_stride;
        }
    };
    int64_t out = s.begin * p.C + c;
    auto token = [&](const ConvRow<T, V>& row) {
        float xt[V], y[V];
        row.get(xt);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            y[v] = conv_pre<W, V>(k, h, xt[v], v);
            if (p.silu) y[v] *= sigmoid_fast(y[v]);
        }
        conv_shift<W, V>(h, xt);
        conv_store<V, true>(p.y, out, y, p.out_bf16);
        out += p.C;
    };
    if (left > 0) load(left);
    while (left > 0) {
        ConvRow<T, V> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        if (left > U) load(left - U);
        if (left >= U) {
#pragma unroll
            for (int u = 0; u < U; ++u) token(now[u]);
        } else {
#pragma unroll
            for (int u = 0; u < U - 1; ++u)
                if (u < left) token(now[u]);
        }
        left -= U;
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
    const int64_t thread = blockIdx.y * blockDim.x + threadIdx.x;
    const int c = conv_channel<V>(thread, p.C);
    if (thread * V >= p.C) return;
    float dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    if (s.begin < s.end || s.last) {
        const ConvWeights<W, V> k(p, c);
        constexpr int U = 2;                      // rows on their way
        float h[W - 1][V], sum[W - 1][V];         // rows before t; the dx of t - W + 1 .. t - 1 so far
        conv_history<T, W, V>(h, p, s, s.begin, c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) sum[j][v] = 0.f;
        const T* x = (const T*)p.x + s.begin * p.x_stride + c;
        const T* dy = (const T*)p.dy + s.begin * p.C + c;
        ConvRow<T, V> nx[U], ng[U];
        int left = (int)(s.hi - s.begin);         // the document's tokens still to load
        auto load = [&]() {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                nx[u].load(x);
                ng[u].load(dy);
                if (--left > 0) { x += p.x_stride; dy += p.C; }
            }
        };
        // token t with its rows; live: before the document's end, own: in this strip
        auto token = [&](const int64_t t, const ConvRow<T, V>& rx, const ConvRow<T, V>& rg) {
            const bool live = t < s.hi, own = t < s.end;
            float g[V], xt[V], dx[V];
            rx.get(xt);
            rg.get(g);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f = g[v];
                if (p.silu) {
                    const float pre = conv_pre<W, V>(k, h, xt[v], v), sig = sigmoid_fast(pre);
                    f *= sig * __builtin_fmaf(pre, 1.f - sig, 1.f);
                }
                f = live ? f : 0.f;
                dx[v] = __builtin_fmaf(k.w[0][v], f, sum[0][v]);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) sum[j][v] = __builtin_fmaf(k.w[j + 1][v], f, sum[j + 1][v]);
                sum[W - 2][v] = k.w[W - 1][v] * f;
                if (own) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][v] = __builtin_fmaf(f, h[j][v], dw[j][v]);
                    dw[W - 1][v] = __builtin_fmaf(f, xt[v], dw[W - 1][v]);
                    dw[W][v] += f;
                }
            }
            conv_shift<W, V>(h, xt);
            const int64_t at = t - (W - 1);       // the row that is complete
            if (at < s.begin && (s.j > 0 || !p.ds0)) return;
            const int64_t r = at - s.hi + (W - 1);   // its row in the final state
            if (r >= 0 && p.dsf) {
                float e[V];
                conv_load<T, V>(e, (const T*)p.dsf + ((int64_t)s.n * (W - 1) + r) * p.C + c);
#pragma unroll
                for (int v = 0; v < V; ++v) dx[v] += e[v];
            }
            if (at >= s.begin) conv_store<V, true>(p.dx, at * p.C + c, dx, p.out_bf16);
            else conv_store<V>(p.ds0, ((int64_t)s.n * (W - 1) + (at - s.lo) + (W - 1)) * p.C + c, dx, sizeof(T) == 2);
        };
        if (left > 0) load();                     // an empty document has no rows
        for (int64_t t = s.begin; t < s.end + W - 1; t += U) {
            ConvRow<T, V> cx[U], cg[U];
#pragma unroll
            for (int u = 0; u < U; ++u) { cx[u] = nx[u]; cg[u] = ng[u]; }
            if (left > 0) load();
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < s.end + W - 1) token(t + u, cx[u], cg[u]);
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
    const int64_t per = (p.C + V - 1) / V;
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
    // a step may run in place, so its threads share no channels
    if (call == kConvDecode ? p.C % 8 == 0 : p.eight) conv_launch<T, W, 8>(p, call, stream);
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
