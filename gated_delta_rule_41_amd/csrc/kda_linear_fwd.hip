// kda_linear_fwd.hip -- the linear rule over packed documents.
//
// With G the inclusive sum of g inside a chunk of 64 tokens and S the state entering it,
//     P_ij = scale e^{G_i - G_j} q_i . k_j  (j <= i)
//     o_i  = sum_j P_ij v_j + scale e^{G_i} S^T q_i
//     S   <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// Nothing in a chunk depends on the chunk before but S, and S only adds up, so the state
// lives in matrix-core accumulators for a whole walk and every decay is a difference of
// sums, at most 1 for g <= 0.
//
// linear_out_kernel: one workgroup (4 waves) walks one document (or one segment of it) for
// one head and 64 value columns; wave c holds the state's columns 16c..16c+15.  Wave w forms
// rows 16w..16w+15 of P and hands them over through LDS; everything else a wave needs of the
// state is its own.  The next chunk's rows are loaded into registers while this one runs.
//
// linear_state_kernel: the state alone, forward or in reverse (the same sum with q, dO and
// weights e^{G_i}), for the segments of long documents and for the backward.
//
// linear_carry_kernel: the states entering the segments of each document, from the
// segments' own sums (a scalar decay composes as plain products).
#include "kda_linear_device.h"

namespace kda {
using namespace lin;

// Chains of one head's value slices sit eight workgroups apart, on one XCD, whose L2 then
// serves the rows that they share.
__device__ __forceinline__ bool chain_slice(int64_t b, int slices, int chains, int& chain, int& slice) {
    const int64_t group = b / (8 * slices);
    const int r = (int)(b % (8 * slices));
    chain = (int)(group * 8 + (r & 7));
    slice = r >> 3;
    return chain < chains;
}

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void linear_out_kernel(LinearParams p) {
    constexpr int C = kLinChunk, LQ = DK + 8, LV = kSlice + 8, LP = C + 8;
    typedef typename V8<T>::t frag;
    __shared__ __align__(32) T sQ[C * LQ];
    __shared__ __align__(32) T sK[C * LQ];
    __shared__ __align__(32) T sV[C * LV];
    __shared__ __align__(32) T sP[C * LP];
    __shared__ __align__(16) double sG[C];
    __shared__ __align__(32) float sW[C];
    __shared__ float sE;

    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, cl = l & 15, qg = l >> 4;
    int chain, slice;
    if (!chain_slice(blockIdx.x, p.dv / kSlice, p.chains, chain, slice)) return;
    const int64_t slot = chain / p.H;
    const int h = chain % p.H, hk = h / (p.H / p.Hk);
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, p.seg_len);
    const int dv = p.dv, col = slice * kSlice + 16 * w;
    if (p.seg_len && rg.lo >= rg.hi) return;

    // the state: block d holds rows 16d + 4qg + i, column col + cl
    f32x4 S[DK / 16];
    {
        const float* s0 = p.s0 ? p.s0 + ((int64_t)(p.seg_len ? slot : rg.n) * p.H + h) * DK * dv + col + cl : nullptr;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[d][i] = s0 ? s0[(int64_t)(16 * d + 4 * qg + i) * dv] : 0.f;
    }

    const T* qp = (const T*)p.q + (rg.lo * p.Hk + hk) * DK;
    const T* kp = (const T*)p.k + (rg.lo * p.Hk + hk) * DK;
    const T* vp = (const T*)p.v + (rg.lo * p.H + h) * dv + slice * kSlice;
    const float* gp = p.g + (p.g_stride ? rg.lo * p.g_stride : 0) + h;
    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * dv;
    const int total = (int)(rg.hi - rg.lo);

    // key blocks above the diagonal that a 32-wide product step still covers stay zero
    for (int x = tid; x < C * LP; x += kThreads) sP[x] = (T)0.f;

    Tile<T, C, DK, kThreads> tq, tk;
    Tile<T, C, kSlice, kThreads> tv;
    float g = 0.f;
    if (total > 0) {
        tq.load(qp, ldk, total, tid);
        tk.load(kp, ldk, total, tid);
        tv.load(vp, ldv, total, tid);
        if (w == 0) g = gp[(int64_t)(l < total ? l : total - 1) * p.g_stride];
    }
    for (int t0 = 0; t0 < total; t0 += C) {
        const int rows = total - t0;
        lds_barrier();   // the last chunk's readers are done
        tq.store(sQ, LQ, rows, tid);
        tk.store(sK, LQ, rows, tid);
        tv.store(sV, LV, rows, tid);
        if (w == 0) {
            const double G = wave_scan(l < rows ? gate_log2(g) : 0.0, l);
            const double Gt = __shfl(G, 63, 64);
            sG[l] = G;
            sW[l] = fast_exp2((float)(Gt - G));
            if (l == 0) sE = fast_exp2((float)Gt);
        }
        if (rows > C) {
            tq.load(qp + (t0 + C) * ldk, ldk, rows - C, tid);
            tk.load(kp + (t0 + C) * ldk, ldk, rows - C, tid);
            tv.load(vp + (t0 + C) * ldv, ldv, rows - C, tid);
            if (w == 0) g = gp[(int64_t)(t0 + C + (l < rows - C ? l : rows - C - 1)) * p.g_stride];
        }
        lds_barrier();

        // P, transposed in the accumulators: row = key 16n + 4qg + i, column = query 16w + cl
        {
            frag qf[DK / 32];
#pragma unroll
            for (int s = 0; s < DK / 32; ++s) qf[s] = lds8(sQ + (16 * w + cl) * LQ + 32 * s + 8 * qg);
            const double gq = sG[16 * w + cl];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n <= w) {
                    f32x4 a = zero4();
#pragma unroll
                    for (int s = 0; s < DK / 32; ++s) a = mma_k32(a, lds8(sK + (16 * n + cl) * LQ + 32 * s + 8 * qg), qf[s]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * n + 4 * qg + i;
                        const float d = fast_exp2((float)(gq - sG[key])) * p.scale;
                        a[i] = key <= 16 * w + cl ? a[i] * d : 0.f;
                    }
                    sts4(sP + (16 * w + cl) * LP + 16 * n + 4 * qg, a);
                }
        }
        // through the entering state; transposed: row = value column, column = token 16m + cl
        f32x4 O[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) O[m] = zero4();
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            const frag sf = pack8<T>(S[2 * s], S[2 * s + 1]);   // bf16 inputs: the state rounded once, for this read only
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const T* q = sQ + (16 * m + cl) * LQ + 32 * s + 4 * qg;
                O[m] = mma_k32(O[m], sf, two4(q, q + 16));
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) O[m] *= fast_exp2((float)sG[16 * m + cl]) * p.scale;
        frag vf[2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) vf[kk] = col_frag(sV, LV, 32 * kk + 8 * qg, 32 * kk + 8 * qg + 4, 16 * w, cl);
        // the state
        const float eC = sE;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) S[d] *= eC;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f32x8 u = widen8(vf[kk]) * lds8(sW + 32 * kk + 8 * qg);
#pragma unroll
            for (int d = 0; d < DK / 16; ++d)
                S[d] = mma_f32x<false>(S[d], u, col_frag(sK, LQ, 32 * kk + 8 * qg, 32 * kk + 8 * qg + 4, 16 * d, cl));
        }
        lds_barrier();   // P is there
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int kk = 0; kk <= m / 2; ++kk)
                O[m] = mma_k32(O[m], vf[kk], lds8(sP + (16 * m + cl) * LP + 32 * kk + 8 * qg));
            const int t = t0 + 16 * m + cl;
            if (t < total) store4(p.o, ((rg.lo + t) * p.H + h) * dv + col + 4 * qg, O[m], p.out_bf16);
        }
    }
    if (p.sfinal && !p.seg_len) {
        float* sf = p.sfinal + ((int64_t)rg.n * p.H + h) * DK * dv + col + cl;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) sf[(int64_t)(16 * d + 4 * qg + i) * dv] = S[d][i];
    }
}

template <typename T, int DK>
__global__ __launch_bounds__(kThreads) void linear_state_kernel(LinearStateParams p) {
    constexpr int C = kLinChunk, LA = DK + 8, LB = kSlice + 8;
    __shared__ __align__(32) T sA[C * LA];
    __shared__ __align__(32) T sB[C * LB];
    __shared__ __align__(32) float sW[C];
    __shared__ float sE;

    const LinearStateDir D = p.dir[blockIdx.y];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, cl = l & 15, qg = l >> 4;
    int chain, slice;
    if (!chain_slice(blockIdx.x, p.dv / kSlice, p.chains, chain, slice)) return;
    const int64_t slot = chain / p.H;
    const int h = chain % p.H, hk = h / (p.H / p.Hk);
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, p.seg_len);
    if (p.seg_len && rg.lo >= rg.hi) return;
    const int dv = p.dv, col = slice * kSlice + 16 * w + 4 * qg;
    const bool rev = D.rev != 0;

    // transposed against linear_out_kernel, for 16-byte stores: block d holds state row
    // 16d + cl, value columns col .. col + 3
    f32x4 S[DK / 16];
    {
        const float* s0 = D.s0 ? D.s0 + ((int64_t)(p.seg_len ? slot : rg.n) * p.H + h) * DK * dv + col : nullptr;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
            S[d] = s0 ? *reinterpret_cast<const f32x4*>(s0 + (int64_t)(16 * d + cl) * dv) : zero4();
    }
    const T* ap = (const T*)D.a + (rg.lo * p.Hk + hk) * DK;
    const T* bp = (const T*)D.b + (rg.lo * p.H + h) * dv + slice * kSlice;
    const float* gp = p.g + (p.g_stride ? rg.lo * p.g_stride : 0) + h;
    const int64_t lda = (int64_t)p.Hk * DK, ldb = (int64_t)p.H * dv;
    const int total = (int)(rg.hi - rg.lo), chunks = (total + C - 1) / C;
    // a block of the document keeps its slot whatever the segments are
    const int64_t block0 = rg.start / kLinBlock + rg.n + (rg.lo - rg.start) / kLinBlock;

    Tile<T, C, DK, kThreads> ta;
    Tile<T, C, kSlice, kThreads> tb;
    float g = 0.f;
    double gsum = 0.0;
    if (chunks > 0) {
        const int t0 = rev ? (chunks - 1) * C : 0, rows = total - t0;
        ta.load(ap + t0 * lda, lda, rows, tid);
        tb.load(bp + t0 * ldb, ldb, rows, tid);
        if (w == 0) g = gp[(int64_t)(t0 + (l < rows ? l : rows - 1)) * p.g_stride];
    }
    for (int x = 0; x < chunks; ++x) {
        const int c = rev ? chunks - 1 - x : x, t0 = c * C, rows = total - t0;
        if (D.border && (rev ? ((c & 1) || x == 0) : !(c & 1))) {
            T* b = (T*)D.border + ((block0 + c / 2) * p.H + h) * DK * dv + col;
#pragma unroll
            for (int d = 0; d < DK / 16; ++d) *reinterpret_cast<typename V4<T>::t*>(b + (int64_t)(16 * d + cl) * dv) = pack4<T>(S[d]);
        }
        lds_barrier();
        ta.store(sA, LA, rows, tid);
        tb.store(sB, LB, rows, tid);
        if (w == 0) {
            const double G = wave_scan(l < rows ? gate_log2(g) : 0.0, l);
            const double Gt = __shfl(G, 63, 64);
            sW[l] = rev ? fast_exp2((float)G) * p.scale : fast_exp2((float)(Gt - G));
            if (l == 0) sE = fast_exp2((float)Gt);
            gsum += Gt;
        }
        if (x + 1 < chunks) {
            const int u0 = rev ? t0 - C : t0 + C, more = total - u0;
            ta.load(ap + u0 * lda, lda, more, tid);
            tb.load(bp + u0 * ldb, ldb, more, tid);
            if (w == 0) g = gp[(int64_t)(u0 + (l < more ? l : more - 1)) * p.g_stride];
        }
        lds_barrier();
        const float eC = sE;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) S[d] *= eC;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int r = 32 * kk + 8 * qg;
            const f32x8 u = widen8(col_frag(sB, LB, r, r + 4, 16 * w, cl)) * lds8(sW + r);
#pragma unroll
            for (int d = 0; d < DK / 16; ++d) S[d] = mma_f32x<true>(S[d], u, col_frag(sA, LA, r, r + 4, 16 * d, cl));
        }
    }
    if (D.last) {
        float* s = D.last + ((int64_t)(p.seg_len ? slot : rg.n) * p.H + h) * DK * dv + col;
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) *reinterpret_cast<f32x4*>(s + (int64_t)(16 * d + cl) * dv) = S[d];
    }
    if (D.decay && slice == 0 && tid == 0) D.decay[slot * p.H + h] = fast_exp2((float)gsum);
}

__global__ __launch_bounds__(kThreads) void linear_carry_kernel(LinearCarryParams p) {
    const LinearCarryDir D = p.dir[blockIdx.y];
    const int parts = p.elems / (4 * kThreads);
    const int part = blockIdx.x % parts;
    const int64_t nh = blockIdx.x / parts;
    const int n = (int)(nh / p.H), h = (int)(nh % p.H);
    int64_t s, e;
    doc_bounds(p.cu, p.seqlen, p.T, n, s, e);
    const int segs = (int)((e - s + p.seg_len - 1) / p.seg_len);
    const int64_t first = s / p.seg_len + n, at = (int64_t)part * 4 * kThreads + 4 * threadIdx.x;
    const int64_t step = (int64_t)p.H * p.elems;
    f32x4 cur = D.s0 ? *reinterpret_cast<const f32x4*>(D.s0 + nh * p.elems + at) : zero4();
    float* st = D.state + (first * p.H + h) * (int64_t)p.elems + at;
    const float* dc = D.decay + first * p.H + h;
    for (int x = 0; x < segs; ++x) {
        const int j = D.rev ? segs - 1 - x : x;
        const f32x4 own = *reinterpret_cast<const f32x4*>(st + j * step);
        const float a = dc[(int64_t)j * p.H];
        *reinterpret_cast<f32x4*>(st + j * step) = cur;
        cur = a * cur + own;
    }
    if (D.last) *reinterpret_cast<f32x4*>(D.last + nh * p.elems + at) = cur;
}

static unsigned grid_of(int chains, int slices) { return (unsigned)((chains + 7) / 8 * 8 * slices); }

template <typename T> static hipError_t out_t(const LinearParams& p, int dk, hipStream_t stream) {
    const dim3 grid(grid_of(p.chains, p.dv / kSlice));
    if (dk == 128) hipLaunchKernelGGL((linear_out_kernel<T, 128>), grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((linear_out_kernel<T, 64>), grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}
hipError_t launch_linear_out(const LinearParams& p, int in_dtype, int dk, hipStream_t stream) {
    return in_dtype == 1 ? out_t<bf16>(p, dk, stream) : out_t<float>(p, dk, stream);
}

template <typename T> static hipError_t states_t(const LinearStateParams& p, int dirs, int dk, hipStream_t stream) {
    const dim3 grid(grid_of(p.chains, p.dv / kSlice), dirs);
    if (dk == 128) hipLaunchKernelGGL((linear_state_kernel<T, 128>), grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((linear_state_kernel<T, 64>), grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}
hipError_t launch_linear_states(const LinearStateParams& p, int dirs, int in_dtype, int dk, hipStream_t stream) {
    return in_dtype == 1 ? states_t<bf16>(p, dirs, dk, stream) : states_t<float>(p, dirs, dk, stream);
}

hipError_t launch_linear_carry(const LinearCarryParams& p, int dirs, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.N * p.H * (p.elems / (4 * kThreads))), dirs);
    hipLaunchKernelGGL(linear_carry_kernel, grid, dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
