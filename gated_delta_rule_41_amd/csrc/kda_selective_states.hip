// kda_selective_states.hip -- states across the segments of a document, forward and in reverse:
// every segment's own sum from a zero state, its share of the gradient of the state that enters
// it, and the carries along the segments.  The own sums walk as the forward does
// (kda_selective.h), without the output's multiply-add and the gate: four instructions an entry
// and token and 19 beside them, 142 us for 67.1M tokens and channels of 16 entries at an
// instruction every four cycles, 173 with second slots.
#include "kda_selective.h"

namespace kda {

// KEEP 0: own sums of all segments but a document's last.  KEEP > 0: of all, and the own state
// before every KEEP tokens with the sum of dt up to there, for the backward.
template <typename T, int S, int KEEP>
__global__ __launch_bounds__(kLayerThreads) void selective_states_kernel(SelectiveParams p) {
    constexpr int U = KEEP ? KEEP : 4;            // tokens a block: their loads are one block ahead
    const Segment s = find_segment(p.cu, p.N, p.seqlen, p.T, p.len, blockIdx.x);
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.y * 4 + (threadIdx.x >> 6)));
    if (s.begin >= s.end || (!KEEP && s.last) || wave >= p.waves) return;
    const Channels ch(p, wave);
    float A2[S], h[S], sum = 0.f;
    load_A<S>(A2, p.A + (int64_t)ch.c * S);
#pragma unroll
    for (int n = 0; n < S; ++n) h[n] = 0.f;
    const float bias = p.bias ? p.bias[ch.c] : 0.f;
    const T* x = (const T*)p.x + s.begin * p.x_stride;
    const T* dt = (const T*)p.dt + s.begin * p.dt_stride;
    UniformRows<T, S> B((const T*)p.B + s.begin * p.b_stride + (int64_t)ch.group * S, p.b_stride);
    T nx[U], nd[U];
    int left = (int)(s.end - s.begin);            // tokens from the block on
    auto load = [&](int count) {                  // the block at x, dt; rows behind the segment are its last
#pragma unroll
        for (int u = 0; u < U; ++u) {
            nx[u] = row_at(x, ch);
            nd[u] = row_at(dt, ch);
            if (u + 1 < count) { x += p.x_stride; dt += p.dt_stride; }
        }
    };
    load(left);
    auto block = [&](auto whole, int count) {
        float d[U], w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            d[u] = step_size(to_f32(nd[u]), bias, p.softplus);
            w[u] = d[u] * to_f32(nx[u]);
        }
        if (whole.value ? left > U : false) load(left - U);
        float part = 0.f;                         // block by block, so that long segments' sums round less
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!whole.value && u >= count) break;
            const UniformRow<T, S> b = B.next(u + 1 < left);
            part += d[u];
#pragma unroll
            for (int n = 0; n < S; ++n) h[n] = __builtin_fmaf(fast_exp2(d[u] * A2[n]), h[n], w[u] * b[n]);
        }
        sum += part;
    };
    int64_t kept = KEEP ? s.lo / U + s.n + (s.begin - s.lo) / U : 0;
    auto keep = [&]() {                           // before every block but the first
        if constexpr (KEEP != 0) {
            ++kept;
            if (left > 0 && ch.valid) {
                store_kept<S>(p.border, kept, p.C, ch.c, h);
                *lane_of(p.bdt + kept * p.C, ch) = sum;
            }
        }
    };
    while (left >= U) {
        block(std::true_type(), U);
        left -= U;
        keep();
    }
    if (left > 0) block(std::false_type(), left);
    if (!ch.valid) return;
    store_kept<S>(p.seg, blockIdx.x, p.C, ch.c, h);
    *lane_of(p.sdt + (int64_t)blockIdx.x * p.C, ch) = sum;
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
    const int64_t z_stride = p.z ? p.z_stride : p.C, at = s.end - 1;
    const T* dy = (const T*)p.dy + at * p.C;
    const T* dt = (const T*)p.dt + at * p.dt_stride;
    const T* z = p.z ? (const T*)p.z + at * z_stride : dy;
    UniformRows<T, S> C((const T*)p.Cm + at * p.c_stride + (int64_t)ch.group * S, -p.c_stride);
    T ng[U], nd[U], nz[U];
    int left = (int)(s.end - s.begin);
    auto load = [&](int count) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ng[u] = row_at(dy, ch);
            nd[u] = row_at(dt, ch);
            nz[u] = row_at(z, ch);
            if (u + 1 < count) { dy -= p.C; dt -= p.dt_stride; z -= z_stride; }
        }
    };
    load(left);
    auto block = [&](auto whole, int count) {
        float d[U], g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            d[u] = step_size(to_f32(nd[u]), bias, p.softplus);
            g[u] = to_f32(ng[u]);
            if (p.z) g[u] *= to_f32(nz[u]) * sigmoid_fast(to_f32(nz[u]));
        }
        if (whole.value ? left > U : false) load(left - U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!whole.value && u >= count) break;
            const UniformRow<T, S> c = C.next(u + 1 < left);
#pragma unroll
            for (int n = 0; n < S; ++n) e[n] = fast_exp2(d[u] * A2[n]) * __builtin_fmaf(g[u], c[n], e[n]);
        }
    };
    for (; left >= U; left -= U) block(std::true_type(), U);
    if (left > 0) block(std::false_type(), left);
    if (ch.valid) store_kept<S>(p.rseg, blockIdx.x, p.C, ch.c, e);
}

// Along a document's segments, one lane for an entry of a channel: what entered the document and the
// segments' own sums become the states entering the segments (or, from the document's end, the
// gradients of the states leaving them).  The waves of a workgroup share a document's segments: each
// goes over its part from zero with the product of its decays, then, from what the parts before it
// make of the entering state, once more and stores.  1366 segments of 512 channels take 34 us with 16
// waves and 101 with one, whose every batch of loads waits for memory.
struct CarryDir {
    const float* first;       // [N,C,S] or nullptr (zero)
    float* seg;
    bool rev;
};
// One wave's part: segments j0 .. j1 - 1 of a document, in the direction's order, h passing through.
template <bool STORE>
__device__ __forceinline__ void carry_part(const SelectiveParams& p, const CarryDir& dir, int64_t first, int64_t per, int j0, int j1,
                                           unsigned i, unsigned c, float A2, float& h, float& decay) {
    // Segments on their way.  The next ones are asked for before these are stored: a wait for loads behind stores
    // would be one for the stores as well.
    constexpr int U = 12;
    const int64_t seg_step = dir.rev ? -per : per, sum_step = dir.rev ? -(int64_t)p.C : p.C;
    const int64_t at = dir.rev ? first - j0 : first + j0;
    const float* from = dir.seg + at * per;       // the next to load, then to store: uniform, i and c are a lane's
    const float* sums = p.sdt + at * p.C;
    float* to = dir.seg + at * per;
    float own[U], sum[U];
    int left = j1 - j0;                           // still to load
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            own[u] = *lane_bytes(from, i * 4);
            sum[u] = *lane_bytes(sums, c * 4);
            if (left > u + 1) { from += seg_step; sums += sum_step; }
        }
    };
    if (left > 0) load();
    for (int j = j0; j < j1; j += U) {
        float a[U], x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = fast_exp2(sum[u] * A2);
            x[u] = own[u];
        }
        left -= U;
        if (left > 0) load();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u >= j1) continue;
            if constexpr (STORE) {
                *lane_bytes(to, i * 4) = h;
                to += seg_step;
            } else {
                decay *= a[u];
            }
            h = __builtin_fmaf(a[u], h, x[u]);
        }
    }
}
constexpr int kCarryWaves = 16;
__global__ __launch_bounds__(64 * kCarryWaves) void selective_carry_kernel(SelectiveParams p, int S) {
    __shared__ float parts[2][kCarryWaves][64];
    const int64_t per = (int64_t)p.C * S;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), waves = blockDim.x >> 6;
    unsigned i = blockIdx.y * 64 + lane;          // [S / 4][C][4]
    const bool valid = i < per;
    i = valid ? i : 0;
    const CarryDir dir = blockIdx.z ? CarryDir{p.dsf, p.rseg, true} : CarryDir{p.s0, p.seg, false};
    const int n = blockIdx.x;
    const unsigned c = i / 4 % (unsigned)p.C, e = c * S + i / 4 / (unsigned)p.C * 4 + i % 4;   // the same entry in [C][S]
    const int64_t lo = doc_start(p.cu, n, p.seqlen, p.T);
    int64_t hi = doc_start(p.cu, n + 1, p.seqlen, p.T);
    hi = hi < lo ? lo : hi;
    const int count = (int)((hi - lo + p.len - 1) / p.len);
    if (count < 2) return;                        // the walk reads the document's own state
    const int64_t slot = lo / p.len + n, first = dir.rev ? slot + count - 1 : slot;
    const float A2 = p.A[e] * kLog2e;
    float h = dir.first && valid ? dir.first[n * per + e] : 0.f;
    // the last segment's own sum is not needed, only what enters it
    const int part = (count - 1 + waves - 1) / waves, j0 = w * part < count - 1 ? w * part : count - 1, j1 = j0 + part < count - 1 ? j0 + part : count - 1;
    if (waves > 1) {
        float own = 0.f, decay = 1.f;
        carry_part<false>(p, dir, first, per, j0, j1, i, c, A2, own, decay);
        parts[0][w][lane] = own;
        parts[1][w][lane] = decay;
        __syncthreads();
        for (int v = 0; v < w; ++v) h = __builtin_fmaf(parts[1][v][lane], h, parts[0][v][lane]);
    }
    float none = 0.f;
    if (valid) carry_part<true>(p, dir, first, per, j0, j1, i, c, A2, h, none);
    if (valid && j0 < j1 && j1 == count - 1) dir.seg[(dir.rev ? first - j1 : first + j1) * per + i] = h;
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
    const int64_t entries = (int64_t)p.C * S;
    // Many waves a document only where there are few documents and channels, and long ones: 4 documents of 171 segments
    // in all x 4096 channels take 39 us with one and 168 with 16, 37 documents 35 and 442, 3 of 83 x 200 channels 7 and 11.
    const int64_t alone = p.N * ((entries + 63) / 64) * (backward ? 2 : 1);
    const int waves = alone <= 1024 && p.T / p.len >= 8 * kCarryWaves ? kCarryWaves : 1;
    hipLaunchKernelGGL(selective_carry_kernel, dim3((unsigned)p.N, (unsigned)((entries + 63) / 64), backward ? 2 : 1), dim3(64 * waves), 0, stream, p, S);
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
