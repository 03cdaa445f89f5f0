// kda_linear_decode.hip -- one token of the linear rule on a resident state:
//     S <- e^g S + k v^T,   o = scale S^T q.
// The step reads and writes the state once (8 dk dv bytes per sequence and head) and a few
// hundred bytes besides, so HBM bounds it.  The layout is kda_decode's: one workgroup (4
// waves) per (sequence, head, 64 value columns), thread (tr, tc) holding state rows
// tr + 16 j and columns 4 tc .. 4 tc + 3, all state loads issued first, loads and stores
// nontemporal (each byte is used once).  Only the output needs a sum over rows, so the
// stores do not wait for it.  256 sequences x 32 heads of 128: 187 us, 5.8 TB/s.
#include "kda_linear_device.h"

namespace kda {
using namespace lin;

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void linear_decode_kernel(LinearDecodeParams p) {
    constexpr int RPT = DK / 16;
    __shared__ float sq[DK], sk[DK];
    __shared__ f32x4 sred[4][16];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, tc = tid & 15, tr = tid >> 4;
    const int slices = p.dv / kSlice;
    const int64_t nh = blockIdx.x / slices;
    const int slice = blockIdx.x % slices;
    const int64_t n = nh / p.H;
    const int h = (int)(nh % p.H), hk = h / (p.H / p.Hk);
    const int col = slice * kSlice + 4 * tc;
    const int64_t base = nh * DK * p.dv + col;

    f32x4 s[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j)
        s[j] = p.s_in ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p.s_in + base + (int64_t)(tr + 16 * j) * p.dv)) : zero4();
    const f32x4 v = unpack4(*reinterpret_cast<const typename V4<T>::t*>((const T*)p.v + nh * p.dv + col));
    const float g = p.g[(p.g_stride ? n * p.g_stride : 0) + h];
    if (tid < DK) {
        sq[tid] = to_f32(((const T*)p.q)[(n * p.Hk + hk) * DK + tid]) * p.scale;
        sk[tid] = to_f32(((const T*)p.k)[(n * p.Hk + hk) * DK + tid]);
    }
    const float a = fast_exp(g);
    __syncthreads();
    f32x4 o = zero4();
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        const int i = tr + 16 * j;
        s[j] = s[j] * a + sk[i] * v;
        o += sq[i] * s[j];
        __builtin_nontemporal_store(s[j], reinterpret_cast<f32x4*>(p.s_out + base + (int64_t)i * p.dv));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[e] += __shfl_xor(o[e], 16, 64);
        o[e] += __shfl_xor(o[e], 32, 64);
    }
    if (l < 16) sred[w][tc] = o;
    __syncthreads();
    if (tid < 16) store4(p.o, nh * p.dv + col, (sred[0][tc] + sred[1][tc]) + (sred[2][tc] + sred[3][tc]), p.out_bf16);
}

template <typename T> static void decode_t(const LinearDecodeParams& p, int dk, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.N * p.H * (p.dv / kSlice)));
    if (dk == 128) hipLaunchKernelGGL((linear_decode_kernel<T, 128>), grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((linear_decode_kernel<T, 64>), grid, dim3(kThreads), 0, stream, p);
}
hipError_t launch_linear_decode(const LinearDecodeParams& p, int in_dtype, int dk, hipStream_t stream) {
    if (p.N == 0) return hipSuccess;
    if (in_dtype == 1) decode_t<bf16>(p, dk, stream);
    else decode_t<float>(p, dk, stream);
    return hipGetLastError();
}

}  // namespace kda
