// kda_linear_bwd.hip -- gradients of the linear rule, parallel over blocks of 128 tokens.
//
// With S the state entering a block, dS the gradient of the state at its end, G the
// inclusive sum of g inside it, D_ij = scale e^{G_i - G_j} (j <= i), w_j = e^{G_n - G_j}:
//     P = (q k^T) o D,   dP = (dO v^T) o D,   A = P o (dO v^T)
//     dq_i = sum_j dP_ij k_j + scale e^{G_i} S dO_i
//     dk_j = sum_i dP_ij q_i + w_j dS v_j
//     dv_j = sum_i P_ij dO_i + w_j dS^T k_j
//     dg_t = sum_{i>=t} (e_i + sum_j A_ij - sum_j A_ji) + sum_{j<t} f_j + e^{G_n} <S, dS>
// where e_i and f_j are q_i . dq_i and k_j . dk_j through S and dS alone.  dg_t is the sum
// over everything that crosses token t; written this way nothing large cancels (the row and
// column sums of A are fp32 products), unlike the sum of q . dq - k . dk to the end of the
// document, whose rounding grows with its length.
//
// linear_dq_kernel and linear_dkv_kernel: one workgroup (8 waves) per block and key head,
// wave w a 16-row block of queries (keys), looping over the key head's value heads, so the
// gradients of shared heads add up in registers in a fixed order.  A wave forms its own rows
// of P and dP in the transposed orientation, in which the accumulators are at once the
// operand of the next product: no exchange between waves.  linear_dg_kernel finishes dg.
#include "kda_linear_device.h"

namespace kda {
using namespace lin;

constexpr int kB = kLinBlock;

// G of the block's 128 tokens (log2 units, 64 bits) into sG; rows past the end keep the last
// sum.  Called by wave 0.
__device__ __forceinline__ void block_gates(double* sG, const float* gp, int64_t stride, int rows, int l) {
    const double x = l < rows ? gate_log2(gp[(int64_t)l * stride]) : 0.0;
    const double y = l + 64 < rows ? gate_log2(gp[(int64_t)(l + 64) * stride]) : 0.0;
    const double a = wave_scan(x, l), b = wave_scan(y, l) + __shfl(a, 63, 64);
    sG[l] = a;
    sG[l + 64] = b;
}

__device__ __forceinline__ float qsum4(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Four elements of a global row as fp32.
template <typename T> __device__ __forceinline__ f32x4 load4f(const T* p) {
    return unpack4(*reinterpret_cast<const typename V4<T>::t*>(p));
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }

// Row `row` of a global matrix as product fragments (zeros where row >= rows).
template <typename T, int D> __device__ __forceinline__ void row_frags(typename V8<T>::t (&f)[D / 32], const T* base, int64_t ld, int row, int rows, int qg) {
    const T* p = base + (int64_t)(row < rows ? row : rows - 1) * ld + 8 * qg;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        f[s] = *reinterpret_cast<const typename V8<T>::t*>(p + 32 * s);
        if (row >= rows) f[s] = typename V8<T>::t{};
    }
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kGradThreads) void linear_dq_kernel(LinearBwdParams p) {
    constexpr int LK = DK + 8, LV = DV + 8;
    typedef typename V8<T>::t frag;
    __shared__ __align__(32) T sK[kB * LK];
    __shared__ __align__(32) T sB[kB * LV];   // the state, then V
    __shared__ __align__(16) double sG[kB];

    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, cl = l & 15, qg = l >> 4;
    const int64_t slot = blockIdx.x / p.Hk;
    const int hk = (int)(blockIdx.x % p.Hk), R = p.H / p.Hk;
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, kB);
    const int rows = (int)(rg.hi - rg.lo);
    if (rows <= 0) return;
    // row blocks are given out so that the waves of one SIMD (w, w + 4) share the causal work evenly
    const int rb = w < 4 ? w : 11 - w, row = 16 * rb + cl;
    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * DV;
    const T* q = (const T*)p.q + (rg.lo * p.Hk + hk) * DK;

    f32x4 dq[DK / 16];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) dq[m] = zero4();
    {
        Tile<T, kB, DK, kGradThreads> t;
        t.load((const T*)p.k + (rg.lo * p.Hk + hk) * DK, ldk, rows, tid);
        t.store(sK, LK, rows, tid);
    }
    for (int r = 0; r < R; ++r) {
        const int h = hk * R + r;
        {
            Tile<T, DK, DV, kGradThreads> t;
            t.load((const T*)p.S + (slot * p.H + h) * DK * DV, DV, DK, tid);
            t.store(sB, LV, DK, tid);
        }
        if (w == 0) block_gates(sG, p.g + (p.g_stride ? rg.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
        frag dof[DV / 32];
        row_frags<T, DV>(dof, (const T*)p.dO + (rg.lo * p.H + h) * DV, ldv, row, rows, qg);
        Tile<T, kB, DV, kGradThreads> tv;
        tv.load((const T*)p.v + (rg.lo * p.H + h) * DV, ldv, rows, tid);
        lds_barrier();
        const double gq = sG[row];
        // through the entering state; row = key channel 16m + 4qg + i, column = query
        const float eq = fast_exp2((float)gq) * p.scale;
        float e = 0.f;
#pragma unroll
        for (int m = 0; m < DK / 16; ++m) {
            f32x4 x = zero4();
#pragma unroll
            for (int s = 0; s < DV / 32; ++s) x = mma_k32(x, lds8(sB + (16 * m + cl) * LV + 32 * s + 8 * qg), dof[s]);
            x *= eq;
            e += dot4(x, load4f(q + (int64_t)(row < rows ? row : 0) * ldk + 16 * m + 4 * qg));
            dq[m] += x;
        }
        e = qsum4(e);
        if (qg == 0 && row < rows) p.e[(int64_t)h * p.T + rg.lo + row] = e;
        lds_barrier();
        tv.store(sB, LV, rows, tid);
        lds_barrier();
        for (int s = 0; s <= rb / 2; ++s) {
            f32x4 a[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * s + u;
                a[u] = zero4();
#pragma unroll
                for (int x = 0; x < DV / 32; ++x) a[u] = mma_k32(a[u], lds8(sB + (16 * n + cl) * LV + 32 * x + 8 * qg), dof[x]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = 16 * n + 4 * qg + i;
                    const float d = fast_exp2((float)(gq - sG[key])) * p.scale;
                    a[u][i] = key <= row ? a[u][i] * d : 0.f;
                }
            }
            const frag f = pack8<T>(a[0], a[1]);   // bf16 inputs: dP rounded to the products' type
#pragma unroll
            for (int m = 0; m < DK / 16; ++m)
                dq[m] = mma_k32(dq[m], col_frag(sK, LK, 32 * s + 4 * qg, 32 * s + 16 + 4 * qg, 16 * m, cl), f);
        }
        lds_barrier();
    }
    if (row < rows)
#pragma unroll
        for (int m = 0; m < DK / 16; ++m)
            store4(p.dq, ((rg.lo + row) * p.Hk + hk) * DK + 16 * m + 4 * qg, dq[m], p.out_bf16);
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kGradThreads) void linear_dkv_kernel(LinearBwdParams p) {
    constexpr int LK = DK + 8, LV = DV + 8;
    constexpr int A = kB * LK > DK * LV ? kB * LK : DK * LV;
    typedef typename V8<T>::t frag;
    __shared__ __align__(32) T sA[A];         // Q, then dS
    __shared__ __align__(32) T sB[kB * LV];   // dO
    __shared__ __align__(16) double sG[kB];
    __shared__ float sRow[8][kB];
    __shared__ float sCol[kB];
    __shared__ float sSum[8];

    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, cl = l & 15, qg = l >> 4;
    const int64_t slot = blockIdx.x / p.Hk;
    const int hk = (int)(blockIdx.x % p.Hk), R = p.H / p.Hk;
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, kB);
    const int rows = (int)(rg.hi - rg.lo);
    if (rows <= 0) return;
    const int rb = w < 4 ? w : 11 - w, key = 16 * rb + cl;
    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * DV;
    const T* k = (const T*)p.k + (rg.lo * p.Hk + hk) * DK;

    frag kf[DK / 32];
    row_frags<T, DK>(kf, k, ldk, key, rows, qg);
    f32x4 dk[DK / 16];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) dk[m] = zero4();
    for (int r = 0; r < R; ++r) {
        const int h = hk * R + r;
        {
            Tile<T, kB, DK, kGradThreads> t;
            t.load((const T*)p.q + (rg.lo * p.Hk + hk) * DK, ldk, rows, tid);
            Tile<T, kB, DV, kGradThreads> u;
            u.load((const T*)p.dO + (rg.lo * p.H + h) * DV, ldv, rows, tid);
            t.store(sA, LK, rows, tid);
            u.store(sB, LV, rows, tid);
        }
        if (w == 0) block_gates(sG, p.g + (p.g_stride ? rg.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
        for (int x = tid; x < 8 * kB; x += kGradThreads) sRow[0][x] = 0.f;
        frag vf[DV / 32];
        row_frags<T, DV>(vf, (const T*)p.v + (rg.lo * p.H + h) * DV, ldv, key, rows, qg);
        f32x4 dv[DV / 16];
#pragma unroll
        for (int m = 0; m < DV / 16; ++m) dv[m] = zero4();
        lds_barrier();
        const double gk = sG[key];
        float colsum = 0.f;
        for (int s = rb / 2; s < (rows + 31) / 32; ++s) {
            f32x4 a[2], b[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * s + u;
                a[u] = b[u] = zero4();
#pragma unroll
                for (int x = 0; x < DK / 32; ++x) a[u] = mma_k32(a[u], lds8(sA + (16 * n + cl) * LK + 32 * x + 8 * qg), kf[x]);
#pragma unroll
                for (int x = 0; x < DV / 32; ++x) b[u] = mma_k32(b[u], lds8(sB + (16 * n + cl) * LV + 32 * x + 8 * qg), vf[x]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int query = 16 * n + 4 * qg + i;
                    const float d = fast_exp2((float)(sG[query] - gk)) * p.scale;
                    const bool on = key <= query;
                    const float P = on ? a[u][i] * d : 0.f;
                    const float x = on ? P * b[u][i] : 0.f;
                    a[u][i] = P;
                    b[u][i] = on ? b[u][i] * d : 0.f;
                    colsum += x;
                    const float rs = row16_sum(x);
                    if (cl == 0) sRow[w][query] = rs;
                }
            }
            const frag fp = pack8<T>(a[0], a[1]), fd = pack8<T>(b[0], b[1]);   // bf16 inputs: P and dP rounded
#pragma unroll
            for (int m = 0; m < DV / 16; ++m)
                dv[m] = mma_k32(dv[m], col_frag(sB, LV, 32 * s + 4 * qg, 32 * s + 16 + 4 * qg, 16 * m, cl), fp);
#pragma unroll
            for (int m = 0; m < DK / 16; ++m)
                dk[m] = mma_k32(dk[m], col_frag(sA, LK, 32 * s + 4 * qg, 32 * s + 16 + 4 * qg, 16 * m, cl), fd);
        }
        colsum = qsum4(colsum);
        if (qg == 0) sCol[key] = colsum;
        float cross = 0.f;
        Tile<T, DK, DV, kGradThreads> td;
        td.load((const T*)p.dS + (slot * p.H + h) * DK * DV, DV, DK, tid);
        {
            Tile<T, DK, DV, kGradThreads> ts;
            ts.load((const T*)p.S + (slot * p.H + h) * DK * DV, DV, DK, tid);
#pragma unroll
            for (int i = 0; i < Tile<T, DK, DV, kGradThreads>::PIECES; ++i) {
                typedef T piece __attribute__((ext_vector_type(16 / sizeof(T))));
                const piece x = __builtin_bit_cast(piece, ts.r[i]), y = __builtin_bit_cast(piece, td.r[i]);
#pragma unroll
                for (int j = 0; j < (int)(16 / sizeof(T)); ++j) cross += to_f32(x[j]) * to_f32(y[j]);
            }
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) cross += __shfl_xor(cross, m, 64);
        if (l == 0) sSum[w] = cross;
        lds_barrier();   // the last readers of Q are done; the sums are there
        td.store(sA, LV, DK, tid);
        if (tid < rows && tid < kB) {
            float x = -sCol[tid];
#pragma unroll
            for (int i = 0; i < 8; ++i) x += sRow[i][tid];
            p.a[(int64_t)h * p.T + rg.lo + tid] = x;
        }
        if (tid == 0) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x += sSum[i];
            p.cross[slot * p.H + h] = x * fast_exp2((float)sG[kB - 1]);
        }
        lds_barrier();
        const float wj = fast_exp2((float)(sG[kB - 1] - gk));
        float f = 0.f;
#pragma unroll
        for (int m = 0; m < DK / 16; ++m) {
            f32x4 x = zero4();
#pragma unroll
            for (int s = 0; s < DV / 32; ++s) x = mma_k32(x, lds8(sA + (16 * m + cl) * LV + 32 * s + 8 * qg), vf[s]);
            x *= wj;
            f += dot4(x, load4f(k + (int64_t)(key < rows ? key : 0) * ldk + 16 * m + 4 * qg));
            dk[m] += x;
        }
        f = qsum4(f);
        if (qg == 0 && key < rows) p.f[(int64_t)h * p.T + rg.lo + key] = f;
#pragma unroll
        for (int m = 0; m < DV / 16; ++m) {
            f32x4 x = zero4();
#pragma unroll
            for (int s = 0; s < DK / 32; ++s) x = mma_k32(x, col_frag(sA, LV, 32 * s + 8 * qg, 32 * s + 8 * qg + 4, 16 * m, cl), kf[s]);
            dv[m] += x * wj;
            if (key < rows) store4(p.dv_out, ((rg.lo + key) * p.H + h) * DV + 16 * m + 4 * qg, dv[m], p.out_bf16);
        }
        lds_barrier();
    }
    if (key < rows)
#pragma unroll
        for (int m = 0; m < DK / 16; ++m)
            store4(p.dk_out, ((rg.lo + key) * p.Hk + hk) * DK + 16 * m + 4 * qg, dk[m], p.out_bf16);
}

// dg of a block, one wave per (block, head): lane l holds tokens l and l + 64.  64-bit sums.
__global__ __launch_bounds__(kThreads) void linear_dg_kernel(LinearBwdParams p) {
    const int l = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= p.blocks * p.H) return;
    const int64_t slot = id / p.H;
    const int h = (int)(id % p.H);
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, kB);
    const int rows = (int)(rg.hi - rg.lo);
    if (rows <= 0) {
        if (p.dg_part && l == 0) p.dg_part[id] = 0.f;
        return;
    }
    const int64_t at = (int64_t)h * p.T + rg.lo;
    double x[2], f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = l + 64 * i;
        x[i] = t < rows ? (double)p.e[at + t] + (double)p.a[at + t] : 0.0;
        f[i] = t < rows ? (double)p.f[at + t] : 0.0;
    }
    const double c = p.cross[id];
    double xs[2], fs[2];
    xs[0] = wave_scan(x[0], l);
    fs[0] = wave_scan(f[0], l);
    xs[1] = wave_scan(x[1], l) + __shfl(xs[0], 63, 64);
    fs[1] = wave_scan(f[1], l) + __shfl(fs[0], 63, 64);
    const double all = __shfl(xs[1], 63, 64);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = l + 64 * i;
        const double d = (all - xs[i] + x[i]) + (fs[i] - f[i]) + c;
        if (t < rows) {
            sum += d;
            if (!p.dg_part) store1(p.dg, (rg.lo + t) * p.H + h, (float)d, p.out_bf16);
        }
    }
    if (p.dg_part) {
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, 64);
        if (l == 0) p.dg_part[id] = (float)sum;
    }
}

// Gate per head: dg[h] is the sum over the blocks, in a fixed order.  One workgroup per head.
__global__ __launch_bounds__(kThreads) void linear_dg_head_kernel(LinearBwdParams p) {
    __shared__ double s[kThreads];
    const int h = blockIdx.x, tid = threadIdx.x;
    double x = 0.0;
    for (int64_t b = tid; b < p.blocks; b += kThreads) x += (double)p.dg_part[b * p.H + h];
    s[tid] = x;
    __syncthreads();
    for (int m = kThreads / 2; m >= 1; m >>= 1) {
        if (tid < m) s[tid] += s[tid + m];
        __syncthreads();
    }
    if (tid == 0) store1(p.dg, h, (float)s[0], p.out_bf16);
}

template <typename T, int DK, int DV> static void grads_t(const LinearBwdParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.blocks * p.Hk));
    hipLaunchKernelGGL((linear_dq_kernel<T, DK, DV>), grid, dim3(kGradThreads), 0, stream, p);
    hipLaunchKernelGGL((linear_dkv_kernel<T, DK, DV>), grid, dim3(kGradThreads), 0, stream, p);
}
template <typename T> static void grads_d(const LinearBwdParams& p, int dk, hipStream_t stream) {
    if (dk == 128) {
        if (p.dv == 128) grads_t<T, 128, 128>(p, stream);
        else grads_t<T, 128, 64>(p, stream);
    } else {
        if (p.dv == 128) grads_t<T, 64, 128>(p, stream);
        else grads_t<T, 64, 64>(p, stream);
    }
}
hipError_t launch_linear_grads(const LinearBwdParams& p, int in_dtype, int dk, hipStream_t stream) {
    if (p.T > 0) {
        if (in_dtype == 1) grads_d<bf16>(p, dk, stream);
        else grads_d<float>(p, dk, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(linear_dg_kernel, dim3((unsigned)((p.blocks * p.H + 3) / 4)), dim3(kThreads), 0, stream, p);
    }
    if (p.dg_part) hipLaunchKernelGGL(linear_dg_head_kernel, dim3(p.H), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
