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
// one head; wave w holds the state's columns [w dv/4, (w + 1) dv/4), so an operand fragment
// of q or k read from LDS serves two products at dv = 128.  Wave w forms rows 16w..16w+15 of
// P and hands them over through LDS; everything else a wave needs of the state is its own.
// The next chunk's rows are loaded into registers while this one runs, and its gates are
// summed by wave 0, which has the least of P.
//
// 131083 tokens x 16 heads of 128, bf16, 512 segments: 491 us, 2.19 GB, 4.5 TB/s (a copy: 5.2).
// Two waves a SIMD issue vector instructions 44% and matrix instructions 33% of that time; at
// 32768 x 32 heads on 8, with a third less to read, it took 251 us against 275 on 32: near both
// bounds.  64 tokens a step are what two workgroups' LDS allows.
//
// linear_state_kernel: the state alone, forward or in reverse (the same sum with q, dO and
// weights e^{G_i}), for the segments of long documents and for the backward.  Own sums of the
// same segments: 255 us, 1.1 GB, 4.3 TB/s.  Both directions of 4 x 8192 x 32 heads with the
// states at the blocks' borders: 355 us, 1.7 GB, 4.8 TB/s.
//
// linear_carry_kernel: the states entering the segments of each document after the first, from
// the segments' own sums (a scalar decay composes as plain products).  In place: a segment's
// slot holds its own sum before and its entering state after.  16 us for 32 segments x 16 heads,
// 8 for 37 documents x 32 heads, about half of it reading and writing the states.
#include "kda_linear_device.h"

namespace kda {
using namespace lin;

// The gates of one chunk, by one wave (lane = token): G (log2 units, 64 bits), and the
// weights of its tokens' writes and of the state.
struct Gates {
    double G[kLinChunk];
    float W[kLinChunk];
    float E;
};
__device__ __forceinline__ double put_gates(Gates& s, float g, int rows, int l, bool rev, float scale) {
    const double G = wave_scan(l < rows ? gate_log2(g) : 0.0), Gt = last_lane(G);
    s.G[l] = G;
    s.W[l] = rev ? fast_exp2((float)G) * scale : fast_exp2((float)(Gt - G));
    if (l == 0) s.E = fast_exp2((float)Gt);
    return Gt;
}
// The gate of token t + lane, for the wave that makes the gates; the other waves' loads read
// nothing (see rows_of).
__device__ __forceinline__ float load_gate(const float* g, int stride, int t, int rows, int l, bool mine) {
    const Buffer b = rows_of(g + (int64_t)t * stride, stride, mine ? rows : 0, kLinChunk, 1);
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, (unsigned)l * stride * 4u, 0, 0));
}

// S += a u over 32 tokens, four blocks of rows at a time, the terms of u in the outer loop: a
// product that adds to the result of the one before it would wait for it.
template <bool U_IS_A, typename T, int NC, int D, typename F>
__device__ __forceinline__ void add_outer(f32x4 (&S)[NC][D], const Split<T> (&u)[NC], F&& rows) {
#pragma unroll
    for (int d0 = 0; d0 < D; d0 += 4) {
        typename V8<T>::t a[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) a[d] = rows(d0 + d);
#pragma unroll
        for (int i = 0; i < Split<T>::TERMS; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int c = 0; c < NC; ++c) S[c][d0 + d] = u[c].template mma<U_IS_A>(i, S[c][d0 + d], a[d]);
    }
}

// O: the type of o.  (As an argument it made a branch around every store, which kept the
// products of a chunk from being scheduled across them.)
template <typename T, typename O, int DK, int DV>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void linear_out_kernel(LinearParams p) {
    constexpr int C = kLinChunk, NC = DV / 64;   // column groups of 16 per wave
    typedef typename V8<T>::t frag;
    __shared__ __align__(32) T sQ[C * DK];
    __shared__ __align__(32) T sK[C * DK];
    __shared__ __align__(32) T sV[C * DV];
    __shared__ __align__(32) T sP[C * C];
    __shared__ __align__(16) float sF[4][C];   // a wave's own decays
    __shared__ __align__(32) Gates gates[2];

    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, cl = l & 15, qg = l >> 4;
    int64_t slot = blockIdx.x / p.H;
    const int h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
    const Range rg = p.longest_first ? longest_range(p.cu, p.N, p.seqlen, p.T, slot, p.seg_len, slot)
                                     : seg_range(p.cu, p.N, p.seqlen, p.T, slot, p.seg_len);
    const int col = 16 * NC * w;
    if (rg.n >= p.N || slot * p.H >= p.chains) return;   // the latter with a malformed cu_seqlens only

    // the state: block d of group c holds rows 16d + 4qg + i, column col + 16c + cl
    f32x4 S[NC][DK / 16];
    {
        // a document's first segment starts from its own state, the others from the carried ones
        const float* s0 = rg.lo > rg.start ? p.seg_state + (slot * p.H + h) * DK * DV + col + cl
                          : p.s0 ? p.s0 + ((int64_t)rg.n * p.H + h) * DK * DV + col + cl : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int d = 0; d < DK / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[c][d][i] = s0 ? s0[(16 * d + 4 * qg + i) * DV + 16 * c] : 0.f;
    }

    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * DV;
    const T* qp = (const T*)p.q + rg.lo * ldk + hk * DK;
    const T* kp = (const T*)p.k + rg.lo * ldk + hk * DK;
    const T* vp = (const T*)p.v + rg.lo * ldv + h * DV;
    const float* gp = p.g + (p.g_stride ? rg.lo * p.g_stride : 0) + h;
    const int total = (int)(rg.hi - rg.lo);

    // key blocks above the diagonal that a 32-wide product step still covers stay zero
    for (int x = tid; x < C * C; x += kThreads) sP[x] = (T)0.f;

    Tile<T, C, DK, kThreads> tq, tk;
    Tile<T, C, DV, kThreads> tv;
    tq.load(qp, ldk, total, tid);
    tk.load(kp, ldk, total, tid);
    tv.load(vp, ldv, total, tid);
    const bool gw = w == 0;
    if (gw) put_gates(gates[0], load_gate(gp, p.g_stride, 0, total, l, true), total, l, false, 0.f);
    float g = load_gate(gp, p.g_stride, C, total - C, l, gw);
    for (int t0 = 0; t0 < total; t0 += C) {
        const int rows = total - t0, cl = opaque(l & 15), qg = opaque(l >> 4);
        const Gates& G = gates[(t0 / C) & 1];
        lds_barrier();   // the last chunk's readers are done
        tq.store(sQ, tid);
        tk.store(sK, tid);
        tv.store(sV, tid);
        const float gn = g;
        g = load_gate(gp, p.g_stride, t0 + 2 * C, rows - 2 * C, l, gw);
        tq.load(qp + (t0 + C) * ldk, ldk, rows - C, tid);
        tk.load(kp + (t0 + C) * ldk, ldk, rows - C, tid);
        tv.load(vp + (t0 + C) * ldv, ldv, rows - C, tid);
        lds_barrier();

        const Lane<T, DK> lk(cl, qg);
        const Lane<T, DV> lv(cl, qg);
        const Lane<T, C> lp(cl, qg);
        constexpr int RK = 16 * DK * sizeof(T), RV = 16 * DV * sizeof(T), RP = 16 * C * sizeof(T);   // bytes of 16 rows
        // P, transposed in the accumulators: row = key 16n + 4qg + i, column = query 16w + cl.
        // Below the diagonal block the decay is split at the last key before the wave's
        // queries, both factors at most 1: one exponential a lane instead of four a block.
        {
            const double gq = G.G[16 * w + cl];
            const double gref = G.G[w ? 16 * w - 1 : 0];
            const float fq = fast_exp2((float)(gq - gref)) * p.scale;
            if (l < 16 * w) sF[w][l] = fast_exp2((float)(gref - G.G[l]));
            frag qf[DK / 32];
#pragma unroll
            for (int s = 0; s < DK / 32; ++s) qf[s] = lk.row(sQ, w * RK, s);
            // two blocks at a time, so that their products do not wait for each other
#pragma unroll
            for (int n0 = 0; n0 < 4; n0 += 2)
                if (n0 <= w) {
                    f32x4 a[2] = {zero4(), zero4()};
#pragma unroll
                    for (int s = 0; s < DK / 32; ++s)
#pragma unroll
                        for (int n = 0; n < 2; ++n) a[n] = mma_k32(a[n], lk.row(sK, (n0 + n) * RK, s), qf[s]);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (n0 + n > w) break;
                        if (n0 + n < w) {
                            a[n] *= lds4(&sF[w][16 * (n0 + n) + 4 * qg]) * fq;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                a[n][i] = keep(a[n][i] * (fast_exp2((float)(gq - G.G[16 * w + 4 * qg + i])) * p.scale), 4 * qg + i <= cl);
                        }
                        put4<T, C>(sP, 16 * w + cl, n0 + n, qg, a[n]);   // bf16 inputs: P rounded to the products' type
                    }
                }
        }
        if (gw) put_gates(gates[(t0 / C + 1) & 1], gn, rows - C, l, false, 0.f);
        // through the entering state; transposed: row = value column, column = token 16m + cl
        f32x4 out[NC][4];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int m = 0; m < 4; ++m) out[c][m] = zero4();
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            frag sf[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) sf[c] = pack8<T>(S[c][2 * s], S[c][2 * s + 1]);   // bf16 inputs: the state rounded, for this read only
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const frag q = lk.perm(sQ, m * RK, s);
#pragma unroll
                for (int c = 0; c < NC; ++c) out[c][m] = mma_k32(out[c][m], sf[c], q);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float e = fast_exp2((float)G.G[16 * m + cl]) * p.scale;
#pragma unroll
            for (int c = 0; c < NC; ++c) out[c][m] *= e;
        }
        frag vf[NC][2];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) vf[c][kk] = lv.col(sV, 2 * kk * RV, w * NC + c);
        lds_barrier();   // P is there
        const Buffer to = rows_of((O*)p.o + (rg.lo + t0) * ldv + h * DV, ldv, rows, C, DV);
        auto store = [&](int m, const f32x4& a, const f32x4& b) __attribute__((always_inline)) {
            const unsigned at = (16 * m + cl) * (unsigned)ldv + col;
            if constexpr (NC == 2) store8<O>(to, at, qg, a, b);
            else store4<O>(to, at + 4 * qg, a);
        };
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int kk = 0; kk <= m / 2; ++kk) {
                const frag f = lp.perm(sP, m * RP, kk);
#pragma unroll
                for (int c = 0; c < NC; ++c) out[c][m] = mma_k32(out[c][m], vf[c][kk], f);
            }
            store(m, out[0][m], out[NC - 1][m]);
        }
        // An infinity or NaN of v is in the last rows, which reach every key, and through the zeros of P in
        // rows before its own: then all rows again, from v's finite values.  131083 tokens x 16 heads take
        // 740 us without this and 758 with it, 37 documents, 16411 tokens, 32 heads on 8 208.7 and 209.7;
        // looking at v itself 764 and 209.5, going over the whole document again where its state ends up
        // infinite or NaN 745 and 214.8.
        f32x4 last = out[0][3];
        if constexpr (NC == 2) last += out[1][3];
        if (__ballot(!(fabsf((last[0] + last[1]) + (last[2] + last[3])) < INFINITY))) {
            __builtin_amdgcn_s_waitcnt(0);
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
                const float e = fast_exp2((float)G.G[16 * m + cl]) * p.scale;
                f32x4 o[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    o[c] = zero4();
#pragma unroll
                    for (int s = 0; s < DK / 32; ++s) o[c] = mma_k32(o[c], pack8<T>(S[c][2 * s], S[c][2 * s + 1]), lk.perm(sQ, m * RK, s));
                    o[c] *= e;
                    for (int kk = 0; kk <= m / 2; ++kk) {
                        const frag x = lv.col(sV, 2 * kk * RV, w * NC + c);
                        o[c] = mma_reaching(o[c], x, lp.perm(sP, m * RP, kk), qg, [&](int key) { return 32 * kk + key <= 16 * m + cl; });
                    }
                }
                store(m, o[0], o[NC - 1]);
            }
        }
        // the state
        const float eC = G.E;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int d = 0; d < DK / 16; ++d) S[c][d] *= eC;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f32x8 wt = join(lds4(G.W + 32 * kk + 4 * qg), lds4(G.W + 32 * kk + 16 + 4 * qg));
            Split<T> u[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) u[c] = Split<T>(widen8(vf[c][kk]) * wt);
            add_outer<false>(S, u, [&](int d) { return lk.col(sK, 2 * kk * RK, d); });
        }
    }
    if (p.sfinal && rg.hi == rg.end) {
        float* sf = p.sfinal + ((int64_t)rg.n * p.H + h) * DK * DV + col + cl;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int d = 0; d < DK / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) sf[(16 * d + 4 * qg + i) * DV + 16 * c] = S[c][d][i];
    }
}

// One workgroup per chain and 64 NC value columns (of a [DK][dv] state).  BORDER: the states at
// the blocks' borders are written too.
template <typename T, int DK, int NC, bool BORDER>
__global__ __launch_bounds__(kThreads, 2) void linear_state_kernel(LinearStateParams p) {
    constexpr int C = kLinChunk, DV = 64 * NC;
    typedef typename V8<T>::t frag;
    __shared__ __align__(32) T sA[C * DK];
    __shared__ __align__(32) T sB[C * DV];
    __shared__ __align__(32) Gates gates[2];

    // The ways of a chain (directions, slices) are eight workgroups apart, on one XCD, whose L2
    // serves the rows that they share; chains without work come last.
    const int ways = p.dirs * (p.dv / DV), way = (int)(blockIdx.x / 8 % ways);
    const int chain = (int)(blockIdx.x / (8 * ways) * 8 + (blockIdx.x & 7));
    if (chain >= p.chains) return;
    const LinearStateDir D = way % p.dirs ? p.dir[1] : p.dir[0];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, cl = l & 15, qg = l >> 4;
    const int64_t slot = chain / p.H;
    const int h = chain % p.H, hk = h / (p.H / p.Hk);
    const int seg_len = segment_length(p.cu, p.N, p.seqlen, p.T, p.seg_len, p.whole_len);
    const Range rg = seg_range(p.cu, p.N, p.seqlen, p.T, slot, seg_len);
    if (rg.n >= p.N) return;
    const bool rev = D.rev != 0;
    const bool head = rev ? rg.hi == rg.end : rg.lo == rg.start, tail = rev ? rg.lo == rg.start : rg.hi == rg.end;
    if (D.decay && tail) return;   // a segment's own sum is for the segments that follow it
    const int col = 16 * NC * w, dv = p.dv, slice = way / p.dirs * DV;

    // transposed against linear_out_kernel, for 16-byte stores: block d of group c holds state
    // row 16d + cl, value columns col + 16c + 4qg + i
    f32x4 S[NC][DK / 16];
    const int lane = cl * dv + slice + col + 4 * qg;
    {
        const float* s0 = D.decay ? nullptr
                          : !head ? D.seg + (slot * p.H + h) * DK * dv + lane
                          : D.s0 ? D.s0 + ((int64_t)rg.n * p.H + h) * DK * dv + lane : nullptr;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int d = 0; d < DK / 16; ++d)
                S[c][d] = s0 ? *reinterpret_cast<const f32x4*>(s0 + 16 * d * dv + 16 * c) : zero4();
    }
    const int64_t lda = (int64_t)p.Hk * DK, ldb = (int64_t)p.H * dv;
    const T* ap = (const T*)D.a + rg.lo * lda + hk * DK;
    const T* bp = (const T*)D.b + rg.lo * ldb + h * dv + slice;
    const float* gp = p.g + (p.g_stride ? rg.lo * p.g_stride : 0) + h;
    const int total = (int)(rg.hi - rg.lo), chunks = (total + C - 1) / C;
    // a block of the document keeps its slot whatever the segments are
    const int64_t block0 = rg.start / kLinBlock + rg.n + (rg.lo - rg.start) / kLinBlock;

    // Chunks go in pairs, one block of the document, of which the second may be behind its end
    // (it adds nothing); in reverse the second comes first.  Rows are loaded two chunks ahead: a
    // chunk takes about as long here as a load does when the memory is busy.
    Tile<T, C, DK, kThreads> ta[2];
    Tile<T, C, DV, kThreads> tb[2];
    float g[2];   // the gates of the chunk after the current one, and of the next one after it
    double gsum = 0.0;
    const bool gw = w == 0;
    const int pairs = (chunks + 1) / 2, dir = rev ? -C : C, first = rev ? (2 * pairs - 1) * C : 0;
    // rows from token t on; none before the document (two chunks past the first in reverse, and
    // in reverse all of an empty document's)
    auto rows_at = [&](int t) { return t < 0 ? 0 : total - t; };
    if (gw) gsum += put_gates(gates[0], load_gate(gp, p.g_stride, first, rows_at(first), l, true), rows_at(first), l, rev, p.scale);
    ta[0].load(ap + first * lda, lda, rows_at(first), tid);
    tb[0].load(bp + first * ldb, ldb, rows_at(first), tid);
    g[1] = load_gate(gp, p.g_stride, first + dir, rows_at(first + dir), l, gw);
    ta[1].load(ap + (first + dir) * lda, lda, rows_at(first + dir), tid);
    tb[1].load(bp + (first + dir) * ldb, ldb, rows_at(first + dir), tid);
    // t0: the chunk's first token; x: 0 for the first of a pair
    auto step = [&](Tile<T, C, DK, kThreads>& ta, Tile<T, C, DV, kThreads>& tb, float& g, const float& gn, int t0, int x) __attribute__((always_inline)) {
        const int cl = opaque(l & 15), qg = opaque(l >> 4);
        const Gates& G = gates[x];
        lds_barrier();   // the last chunk's readers are done
        ta.store(sA, tid);
        tb.store(sB, tid);
        if constexpr (BORDER)
            if (x == 0) {
                T* b = (T*)D.border + ((block0 + t0 / kLinBlock) * p.H + h) * DK * dv;
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int d = 0; d < DK / 16; ++d) *reinterpret_cast<f32x4*>(b + lane + 16 * d * dv + 16 * c) = S[c][d];
                } else if constexpr (NC == 2) {
#pragma unroll
                    for (int d = 0; d < DK / 16; ++d)
                        *reinterpret_cast<u32x4*>(b + (16 * d + cl) * dv + slice + col + trade_col(qg)) = trade_bf16(S[0][d], S[1][d]);
                } else {   // one group of columns: the trade is between two blocks of rows
#pragma unroll
                    for (int d = 0; d < DK / 16; d += 2)
                        *reinterpret_cast<u32x4*>(b + (16 * (d + (qg & 1)) + cl) * dv + slice + col + 8 * (qg >> 1)) = trade_bf16(S[0][d], S[0][d + 1]);
                }
            }
        const int t2 = t0 + 2 * dir, rows2 = rows_at(t2);
        g = load_gate(gp, p.g_stride, t2, rows2, l, gw);
        ta.load(ap + t2 * lda, lda, rows2, tid);
        tb.load(bp + t2 * ldb, ldb, rows2, tid);
        lds_barrier();
        const Lane<T, DK> la(cl, qg);
        const Lane<T, DV> lb(cl, qg);
        if (gw) {
            gsum += put_gates(gates[1 - x], gn, rows_at(t0 + dir), l, rev, p.scale);
        }
        const float eC = G.E;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int d = 0; d < DK / 16; ++d) S[c][d] *= eC;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const f32x8 wt = join(lds4(G.W + 32 * kk + 4 * qg), lds4(G.W + 32 * kk + 16 + 4 * qg));
            Split<T> u[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) u[c] = Split<T>(widen8(lb.col(sB, 2 * kk * 16 * DV * (int)sizeof(T), w * NC + c)) * wt);
            add_outer<true>(S, u, [&](int d) { return la.col(sA, 2 * kk * 16 * DK * (int)sizeof(T), d); });
        }
    };
    for (int y = 0; y < pairs; ++y) {
        const int t0 = first + 2 * y * dir;
        step(ta[0], tb[0], g[0], g[1], t0, 0);
        step(ta[1], tb[1], g[1], g[0], t0 + dir, 1);
    }
    float* s = D.decay ? D.seg + (slot * p.H + h) * DK * dv + lane
               : D.last && tail ? D.last + ((int64_t)rg.n * p.H + h) * DK * dv + lane : nullptr;
    if (s) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int d = 0; d < DK / 16; ++d) *reinterpret_cast<f32x4*>(s + 16 * d * dv + 16 * c) = S[c][d];
    }
    if (D.decay && slice == 0 && tid == 0) D.decay[slot * p.H + h] = fast_exp2((float)gsum);
}

// V vectors of four elements per thread.
template <int V>
__global__ __launch_bounds__(kThreads) void linear_carry_kernel(LinearCarryParams p) {
    const LinearCarryDir D = p.dir[blockIdx.y];
    const int parts = p.elems / (4 * V * kThreads);
    const int part = blockIdx.x % parts;
    const int64_t nh = blockIdx.x / parts;
    const int n = (int)(nh / p.H), h = (int)(nh % p.H);
    int64_t s, e;
    doc_bounds(p.cu, p.seqlen, p.T, n, s, e);
    const int seg_len = segment_length(p.cu, p.N, p.seqlen, p.T, p.seg_len, p.whole_len);
    const int segs = (int)((e - s + seg_len - 1) / seg_len);
    if (segs < 2) return;
    const int64_t first = segments_before(p.cu, p.seqlen, p.T, seg_len, n), at = ((int64_t)part * V * kThreads + threadIdx.x) * 4;
    if (first + segs > p.slots) return;   // a malformed cu_seqlens only
    const int64_t step = D.rev ? -(int64_t)p.H * p.elems : (int64_t)p.H * p.elems;
    const int64_t from = first + (D.rev ? segs - 1 : 0);
    float* st = D.seg + (from * p.H + h) * (int64_t)p.elems + at;
    const float* dc = D.decay + from * p.H + h;
    f32x4 cur[V], own[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        cur[i] = D.s0 ? *reinterpret_cast<const f32x4*>(D.s0 + nh * p.elems + at + i * 4 * kThreads) : zero4();
        own[i] = *reinterpret_cast<const f32x4*>(st + i * 4 * kThreads);
    }
    for (int x = 1; x < segs; ++x) {
        st += step;
        const float a = *dc;
        dc += D.rev ? -p.H : p.H;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f32x4* at_i = reinterpret_cast<f32x4*>(st + i * 4 * kThreads);
            const f32x4 next = x + 1 < segs ? *at_i : zero4();
            cur[i] = a * cur[i] + own[i];
            *at_i = cur[i];
            own[i] = next;
        }
    }
}

template <typename T, typename O> static hipError_t out_t(const LinearParams& p, int dk, hipStream_t stream) {
    const dim3 grid((unsigned)p.chains);
    if (dk == 128) {
        if (p.dv == 128) hipLaunchKernelGGL((linear_out_kernel<T, O, 128, 128>), grid, dim3(kThreads), 0, stream, p);
        else hipLaunchKernelGGL((linear_out_kernel<T, O, 128, 64>), grid, dim3(kThreads), 0, stream, p);
    } else {
        if (p.dv == 128) hipLaunchKernelGGL((linear_out_kernel<T, O, 64, 128>), grid, dim3(kThreads), 0, stream, p);
        else hipLaunchKernelGGL((linear_out_kernel<T, O, 64, 64>), grid, dim3(kThreads), 0, stream, p);
    }
    return hipGetLastError();
}
hipError_t launch_linear_out(const LinearParams& p, int in_dtype, int dk, hipStream_t stream) {
    if (in_dtype == 1) return p.out_bf16 ? out_t<bf16, bf16>(p, dk, stream) : out_t<bf16, float>(p, dk, stream);
    return p.out_bf16 ? out_t<float, bf16>(p, dk, stream) : out_t<float, float>(p, dk, stream);
}

template <typename T, int DK, int NC> static void states_n(const LinearStateParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)p.chains + 7) / 8 * 8 * p.dirs * (p.dv / (64 * NC))));
    if (p.dir[0].border) hipLaunchKernelGGL((linear_state_kernel<T, DK, NC, true>), grid, dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((linear_state_kernel<T, DK, NC, false>), grid, dim3(kThreads), 0, stream, p);
}
template <typename T, int DK> static void states_d(const LinearStateParams& p, hipStream_t stream) {
    // bf16: 128 columns a workgroup halve the reads of `a` from LDS (forward of 131083 tokens x 16
    // heads 814 -> 771 us, backward of 4 documents x 32 heads 1161 -> 1135), as long as whole
    // documents give a workgroup a compute unit, or segments two (backward of 8192 tokens x 8
    // heads with one: 116 -> 119).  fp32: the matrix unit bounds it, and its 128 columns leave
    // room for fewer workgroups (backward of 8 documents x 32 heads 1064 -> 1117).
    if constexpr (sizeof(T) == 2) {
        const bool cut = p.seg_len && p.T / p.seg_len > p.N;
        const int64_t walks = (cut ? p.T / p.seg_len : p.N) * p.H * p.dirs;
        if (p.dv == 128 && walks >= (cut ? kWalkTarget : kWalkTarget / 2)) return states_n<T, DK, 2>(p, stream);
    }
    states_n<T, DK, 1>(p, stream);
}
template <typename T> static hipError_t states_t(const LinearStateParams& p, int dk, hipStream_t stream) {
    if (dk == 128) states_d<T, 128>(p, stream);
    else states_d<T, 64>(p, stream);
    return hipGetLastError();
}
hipError_t launch_linear_states(const LinearStateParams& p, int in_dtype, int dk, hipStream_t stream) {
    return in_dtype == 1 ? states_t<bf16>(p, dk, stream) : states_t<float>(p, dk, stream);
}

hipError_t launch_linear_carry(const LinearCarryParams& p, int dirs, hipStream_t stream) {
    // many documents: most workgroups have nothing to do, so there are fewer of them
    const int64_t nh = (int64_t)p.N * p.H, units = nh * (p.elems / (4 * kThreads));
    if (nh < 256) hipLaunchKernelGGL(linear_carry_kernel<1>, dim3((unsigned)units, dirs), dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL(linear_carry_kernel<4>, dim3((unsigned)(units / 4), dirs), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
