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
// linear_grads_kernel: one workgroup (8 waves) per block, key head and role: dq (with e and the
// row sums of A), dk (with f and its column sums) or dv (with <S, dS>), wave w a 16-row block
// of queries or keys.  Each role loops over the key head's value heads in the same order, so
// that the L2 still has what another role has read (with dv's value heads side by side instead
// 32768 tokens x 32 heads on 16 key heads took 1495 us, like this 1237), and the gradients of shared
// heads add up in registers in a fixed order.  Where that leaves too few workgroups, the value
// heads are divided among `parts` of them, whose sums linear_parts_kernel adds, again in a
// fixed order.  A wave forms its own rows of P or dP in the transposed orientation, in which the
// accumulators are at once the operand of the next product: no exchange between waves, at the
// price of forming dP twice and P twice.  One role needs two 128-row tiles in LDS and fits 128
// registers, so two workgroups share a compute unit and one computes while the other loads;
// the three roles of a block are issued eight workgroups apart, on one XCD, whose L2 serves the
// rows that they share.  At 4 x 8192 tokens x 32 heads, bf16, it takes 655 us and moves 2.46 GB
// (3.8 TB/s, 73% of a copy's rate; matrix instructions issue 20% of the time, vector instructions
// 43%, LDS is busy 31%).  None of them is at its limit: latency bounds it, two workgroups in turn
// through loads, products and stores.
// (One kernel for dk and dv at 255 registers, one workgroup a compute unit, took 620 us, and dq
// beside it 461.)
// linear_dg_kernel finishes dg.
#include "kda_linear_device.h"

namespace kda {
using namespace lin;

constexpr int kB = kLinBlock;

// G of the block's 128 tokens (log2 units, 64 bits) into sG; rows past the end keep the last
// sum.  Called by wave 0.
__device__ __forceinline__ void block_gates(double* sG, const float* gp, int64_t stride, int rows, int l) {
    const double x = l < rows ? gate_log2(gp[(int64_t)l * stride]) : 0.0;
    const double y = l + 64 < rows ? gate_log2(gp[(int64_t)(l + 64) * stride]) : 0.0;
    const double a = wave_scan(x), b = wave_scan(y) + last_lane(a);
    sG[l] = a;
    sG[l + 64] = b;
}

__device__ __forceinline__ float qsum4(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Elements 4 hi .. 4 hi + 3 of a fragment as fp32: of a row fragment in the k order of
// stacked accumulator blocks, what block 2 s + hi holds of that row.
__device__ __forceinline__ f32x4 half4(bf16x8 x, int hi) {
    return hi ? unpack4(__builtin_shufflevector(x, x, 4, 5, 6, 7)) : unpack4(__builtin_shufflevector(x, x, 0, 1, 2, 3));
}
__device__ __forceinline__ f32x4 half4(f32x8 x, int hi) {
    return hi ? __builtin_shufflevector(x, x, 4, 5, 6, 7) : __builtin_shufflevector(x, x, 0, 1, 2, 3);
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3]; }

// Eight elements at a byte offset.
template <typename T> __device__ __forceinline__ typename V8<T>::t load_frag(Buffer b, unsigned off) {
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(bf16x8, load16(b, off));
    else return join(__builtin_bit_cast(f32x4, load16(b, off)), __builtin_bit_cast(f32x4, load16(b, off + 16)));
}

// Row `row` of a global matrix as product fragments (zeros where row >= rows).
template <typename T, int D> __device__ __forceinline__ void row_frags(typename V8<T>::t (&f)[D / 32], const T* base, int64_t ld, int row, int rows, int qg) {
    const Buffer b = rows_of(base, ld, rows, kB, D);
    const unsigned off = ((unsigned)row * (unsigned)ld + 8 * qg) * sizeof(T);
#pragma unroll
    for (int s = 0; s < D / 32; ++s) f[s] = load_frag<T>(b, off + 32 * s * sizeof(T));
}
// The same row in the k order of two stacked accumulator blocks.
template <typename T, int D> __device__ __forceinline__ void row_perms(typename V8<T>::t (&f)[D / 32], const T* base, int64_t ld, int row, int rows, int qg) {
    const Buffer b = rows_of(base, ld, rows, kB, D);
    if constexpr (sizeof(T) == 2) {
        const unsigned off = ((unsigned)row * (unsigned)ld + trade_col(qg)) * 2;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            const u32x4 x = load16(b, off + 64 * s);
            f[s] = __builtin_bit_cast(bf16x8, trade(u32x2{x[0], x[1]}, u32x2{x[2], x[3]}));
        }
    } else {
        const unsigned off = ((unsigned)row * (unsigned)ld + 4 * qg) * 4;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) f[s] = join(__builtin_bit_cast(f32x4, load16(b, off + 128 * s)), __builtin_bit_cast(f32x4, load16(b, off + 128 * s + 64)));
    }
}

// What a role's workgroup knows of its block.
struct Task {
    int64_t slot, lo;
    int rows, hk;
    int h0, h1;        // its value heads
    float* sums;       // where dq or dk goes if other workgroups have the key head's other value heads
};

// LDS of a role: two tiles of 128 rows (the second one also holds the state), the gates, and
// the waves' own decays.
template <typename T, int DK, int DV> struct GradTiles {
    static constexpr int A = kB * (DK > DV ? DK : DV), D = DK * DV, B = A > D ? A : D;
    __align__(32) T a[A];
    __align__(32) T b[B];
    __align__(16) double G[kB];
    __align__(16) float F[8][kB];
    float sum[8];
    __align__(16) unsigned odd[8];   // whether a wave's part of the masked tile holds infinities or NaN
};

// Infinities and NaN of the tile whose rows a mask keeps from some of a block's results.  The zeros of
// the mask times one of them would be NaN, so the tile gets its finite values alone (put_finite), and
// in the end what the others reach becomes NaN (odd_results).  Both are rare, and the second reads
// memory again rather than keep anything in between.  Looking for them costs 4 x 8192 tokens x 32 heads
// 1006 -> 1017 us, 32 heads on 16 1084 -> 1099 (looked for and taken out of LDS after the barrier: 1124).
template <typename S, typename T, int COLS>
__device__ __forceinline__ void put_finite(S& s, const Tile<T, kB, COLS, kGradThreads>& t, T* tile, int tid, int w) {
    t.store(tile, tid);
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < t.PIECES; ++i) x = probe<T>(t.r[i], x);
    const bool any = __ballot(x != 0.f) != 0;
    s.odd[w] = any;   // by every lane: no branch
    if (any) {
        Tile<T, kB, COLS, kGradThreads> f;
#pragma unroll
        for (int i = 0; i < t.PIECES; ++i) f.r[i] = finite_piece<T>(t.r[i]);
        f.store(tile, tid);
    }
}
// After a barrier; the same for the whole workgroup.
template <typename S> __device__ __forceinline__ bool any_odd(const S& s) {
    const u32x4 o = *reinterpret_cast<const u32x4*>(s.odd) | *reinterpret_cast<const u32x4*>(s.odd + 4);
    return __builtin_amdgcn_readfirstlane(o[0] | o[1] | o[2] | o[3]) != 0;
}
// NaN in the results (in the accumulator layout, column = the lane's row of the block) that the rows
// 32 x0 .. 32 x1 - 1 of `base` reach; returns how many reach the lane's row.
template <typename T, int COLS, typename F>
__device__ __forceinline__ float odd_results(f32x4 (&y)[COLS / 16], const T* base, int64_t ld, int rows, int x0, int x1, int cl, int qg, F&& reach) {
    const Buffer b = rows_of(base, ld, rows, kB, COLS);
    float all = 0.f;
#pragma unroll
    for (int m = 0; m < COLS / 16; ++m) {
        f32x4 n = zero4();
#pragma unroll 1
        for (int x = x0; x < x1; ++x) {
            typename V8<T>::t f;
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = load_one<T>(b, (32 * x + (e < 4 ? 0 : 12) + 4 * qg + e) * (unsigned)ld + 16 * m + cl);
            n += odd_count(f, qg, [&](int row) { return reach(32 * x + row); });
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[m][i] = n[i] > 0.f ? __builtin_nanf("") : y[m][i];
        all += (n[0] + n[1]) + (n[2] + n[3]);
    }
    return qsum4(all);
}

// Wave w's 16 rows of a block: row blocks are given out so that the waves of one SIMD (w and
// w + 4) share the causal work evenly.
__device__ __forceinline__ int row_block(int w) { return w < 4 ? w : 11 - w; }

template <typename T, int DK, int DV, bool GROUPED>
__device__ __forceinline__ void dq_role(const LinearBwdParams& p, const Task& t, GradTiles<T, DK, DV>& s) {
    typedef typename V8<T>::t frag;
    constexpr int RK = 16 * DK * sizeof(T), RV = 16 * DV * sizeof(T);   // bytes of 16 rows
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rb = row_block(w), rows = t.rows;
    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * DV;
    const T* q = (const T*)p.q + t.lo * ldk + t.hk * DK;

    f32x4 dq[DK / 16];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) dq[m] = zero4();
    for (int h = t.h0; h < (GROUPED ? t.h1 : t.h0 + 1); ++h) {
        const bool first = !GROUPED || h == t.h0;
        const int tid = GROUPED ? opaque(threadIdx.x) : threadIdx.x, l = tid & 63, cl = l & 15, qg = l >> 4, row = 16 * rb + cl;
        // every load of the step is issued before the first wait
        Tile<T, DK, DV, kGradThreads> ts;
        ts.load((const T*)p.S + (t.slot * p.H + h) * DK * DV, DV, DK, tid);
        frag dof[DV / 32], qf[DK / 32];
        row_frags<T, DV>(dof, (const T*)p.dO + t.lo * ldv + h * DV, ldv, row, rows, qg);
        if constexpr (!GROUPED) row_perms<T, DK>(qf, q, ldk, row, rows, qg);
        Tile<T, kB, DV, kGradThreads> tv;
        if constexpr (!GROUPED) tv.load((const T*)p.v + t.lo * ldv + h * DV, ldv, rows, tid);
        if (first) {
            Tile<T, kB, DK, kGradThreads> tk;
            tk.load((const T*)p.k + t.lo * ldk + t.hk * DK, ldk, rows, tid);
            if (w == 0) block_gates(s.G, p.g + (p.g_stride ? t.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
            ts.store(s.b, tid);
            put_finite(s, tk, s.a, tid, w);
        } else {
            if (w == 0) block_gates(s.G, p.g + (p.g_stride ? t.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
            ts.store(s.b, tid);
        }
        if constexpr (GROUPED) row_perms<T, DK>(qf, q, ldk, row, rows, qg);
        lds_barrier();
        // through the entering state; row = key channel 16m + 4qg + i, column = query
        const Lane<T, DK> lk(cl, qg);
        const Lane<T, DV> lv(cl, qg);
        const double gq = s.G[row];
        const float eq = fast_exp2((float)gq) * p.scale;
        float e = 0.f;   // q . dq through the state, then the row sums of A
#pragma unroll
        for (int m = 0; m < DK / 16; m += 2) {
            f32x4 x[2] = {zero4(), zero4()};
#pragma unroll
            for (int y = 0; y < DV / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) x[u] = mma_k32(x[u], lv.row(s.b, (m + u) * RV, y), dof[y]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[u] *= eq;
                e += dot4(x[u], half4(qf[m / 2], u));
                dq[m + u] += x[u];
            }
            __builtin_amdgcn_sched_barrier(0);   // keeps the reads ahead of it to two blocks' registers
        }
        // with the gradient of the heads before in registers there is no room for it earlier
        if constexpr (GROUPED) tv.load((const T*)p.v + t.lo * ldv + h * DV, ldv, rows, tid);
        lds_barrier();   // the last readers of the state are done
        tv.store(s.b, tid);
        // Below the diagonal block the decay is split at the last key before the wave's
        // queries, both factors at most 1: two exponentials a lane instead of four a block.
        const double gref = s.G[rb ? 16 * rb - 1 : 0];
        const float fq = fast_exp2((float)(gq - gref)) * p.scale;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (l + 64 * i < 16 * rb) s.F[w][l + 64 * i] = fast_exp2((float)(gref - s.G[l + 64 * i]));
        lds_barrier();
        for (int x = 0; x <= rb / 2; ++x) {
            // the products of both blocks side by side, so that none waits for the one before it
            f32x4 a[2] = {zero4(), zero4()}, b[2] = {zero4(), zero4()};
#pragma unroll
            for (int y = 0; y < DV / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) a[u] = mma_k32(a[u], lv.row(s.b, (2 * x + u) * RV, y), dof[y]);
#pragma unroll
            for (int y = 0; y < DK / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) b[u] = mma_k32(b[u], lk.perm(s.a, (2 * x + u) * RK, y), qf[y]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * x + u;
                if (n < rb) {
                    a[u] *= lds4(&s.F[w][16 * n + 4 * qg]) * fq;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * n + 4 * qg + i;
                        const bool on = key <= row;
                        a[u][i] = keep(a[u][i] * (fast_exp2((float)(gq - s.G[key])) * p.scale), on);
                        b[u][i] = keep(b[u][i], on);
                    }
                }
                e += dot4(a[u], b[u]);   // A_ij = dP_ij q_i . k_j
            }
            const frag f = pack8<T>(a[0], a[1]);   // bf16 inputs: dP rounded to the products' type
#pragma unroll
            for (int m = 0; m < DK / 16; ++m) dq[m] = mma_k32(dq[m], lk.col(s.a, 2 * x * RK, m), f);
        }
        e = qsum4(e);
        if (qg == 0 && row < rows) p.e[(int64_t)h * p.T + t.lo + row] = e;
        lds_barrier();
    }
    const int l = threadIdx.x & 63, row = 16 * rb + (l & 15);
    if (any_odd(s)) {
        const float n = odd_results<T, DK>(dq, (const T*)p.k + t.lo * ldk + t.hk * DK, ldk, rows, 0, rb / 2 + 1, l & 15, l >> 4, [&](int key) { return key <= row; });
        if (n > 0.f && row < rows)   // their A as well
            for (int h = t.h0; h < t.h1; ++h) p.e[(int64_t)h * p.T + t.lo + row] = NAN;
    }
    if (GROUPED && t.sums) store_row<DK>(t.sums, t.lo * ldk + t.hk * DK, ldk, rows, kB, row, l >> 4, dq, 0);
    else store_row<DK>(p.dq, t.lo * ldk + t.hk * DK, ldk, rows, kB, row, l >> 4, dq, p.out_bf16);
}

template <typename T, int DK, int DV, bool GROUPED>
__device__ __forceinline__ void dk_role(const LinearBwdParams& p, const Task& t, GradTiles<T, DK, DV>& s) {
    typedef typename V8<T>::t frag;
    constexpr int RK = 16 * DK * sizeof(T), RV = 16 * DV * sizeof(T);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rb = row_block(w), rows = t.rows;
    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * DV;
    const T* k = (const T*)p.k + t.lo * ldk + t.hk * DK;

    f32x4 dk[DK / 16];
#pragma unroll
    for (int m = 0; m < DK / 16; ++m) dk[m] = zero4();
    for (int h = t.h0; h < (GROUPED ? t.h1 : t.h0 + 1); ++h) {
        const bool first = !GROUPED || h == t.h0;
        const int tid = GROUPED ? opaque(threadIdx.x) : threadIdx.x, l = tid & 63, cl = l & 15, qg = l >> 4, key = 16 * rb + cl;
        Tile<T, DK, DV, kGradThreads> td;
        td.load((const T*)p.dS + (t.slot * p.H + h) * DK * DV, DV, DK, tid);
        frag vf[DV / 32], kf[DK / 32];
        row_frags<T, DV>(vf, (const T*)p.v + t.lo * ldv + h * DV, ldv, key, rows, qg);
        if constexpr (!GROUPED) row_perms<T, DK>(kf, k, ldk, key, rows, qg);
        Tile<T, kB, DV, kGradThreads> to;
        if constexpr (!GROUPED) to.load((const T*)p.dO + t.lo * ldv + h * DV, ldv, rows, tid);
        if (first) {
            Tile<T, kB, DK, kGradThreads> tq;
            tq.load((const T*)p.q + t.lo * ldk + t.hk * DK, ldk, rows, tid);
            if (w == 0) block_gates(s.G, p.g + (p.g_stride ? t.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
            td.store(s.b, tid);
            put_finite(s, tq, s.a, tid, w);
        } else {
            if (w == 0) block_gates(s.G, p.g + (p.g_stride ? t.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
            td.store(s.b, tid);
        }
        if constexpr (GROUPED) row_perms<T, DK>(kf, k, ldk, key, rows, qg);
        lds_barrier();
        // through the state's gradient; row = key channel, column = key
        const Lane<T, DK> lk(cl, qg);
        const Lane<T, DV> lv(cl, qg);
        const double gk = s.G[key];
        const float wj = fast_exp2((float)(s.G[kB - 1] - gk));
        float f = 0.f;
#pragma unroll
        for (int m = 0; m < DK / 16; m += 2) {
            f32x4 x[2] = {zero4(), zero4()};
#pragma unroll
            for (int y = 0; y < DV / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) x[u] = mma_k32(x[u], lv.row(s.b, (m + u) * RV, y), vf[y]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[u] *= wj;
                f += dot4(x[u], half4(kf[m / 2], u));
                dk[m + u] += x[u];
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        f = qsum4(f);
        if (qg == 0 && key < rows) p.f[(int64_t)h * p.T + t.lo + key] = f;
        if constexpr (GROUPED) to.load((const T*)p.dO + t.lo * ldv + h * DV, ldv, rows, tid);
        lds_barrier();   // the last readers of dS are done
        to.store(s.b, tid);
        // Above the diagonal block the decay is split at the wave's last key.
        const double gref = s.G[16 * rb + 15];
        const float fk = fast_exp2((float)(gref - gk)) * p.scale;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (l + 64 * i >= 16 * rb + 16) s.F[w][l + 64 * i] = fast_exp2((float)(s.G[l + 64 * i] - gref));
        lds_barrier();
        float colsum = 0.f;
        for (int x = rb / 2; x < (rows + 31) / 32; ++x) {
            f32x4 a[2] = {zero4(), zero4()}, b[2] = {zero4(), zero4()};
#pragma unroll
            for (int y = 0; y < DK / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) a[u] = mma_k32(a[u], lk.perm(s.a, (2 * x + u) * RK, y), kf[y]);
#pragma unroll
            for (int y = 0; y < DV / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) b[u] = mma_k32(b[u], lv.row(s.b, (2 * x + u) * RV, y), vf[y]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * x + u;
                if (n > rb) {
                    b[u] *= lds4(&s.F[w][16 * n + 4 * qg]) * fk;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int query = 16 * n + 4 * qg + i;
                        const bool on = key <= query;
                        b[u][i] = keep(b[u][i] * (fast_exp2((float)(s.G[query] - gk)) * p.scale), on);
                        a[u][i] = keep(a[u][i], on);
                    }
                }
                colsum += dot4(a[u], b[u]);   // A_ij = q_i . k_j dP_ij
            }
            const frag f = pack8<T>(b[0], b[1]);   // bf16 inputs: dP rounded to the products' type
#pragma unroll
            for (int m = 0; m < DK / 16; ++m) dk[m] = mma_k32(dk[m], lk.col(s.a, 2 * x * RK, m), f);
        }
        colsum = qsum4(colsum);
        if (qg == 0 && key < rows) p.a[(int64_t)h * p.T + t.lo + key] = colsum;
        lds_barrier();
    }
    const int l = threadIdx.x & 63, key = 16 * rb + (l & 15);
    if (any_odd(s)) {
        const float n = odd_results<T, DK>(dk, (const T*)p.q + t.lo * ldk + t.hk * DK, ldk, rows, rb / 2, kB / 32, l & 15, l >> 4, [&](int query) { return key <= query; });
        if (n > 0.f && key < rows)
            for (int h = t.h0; h < t.h1; ++h) p.a[(int64_t)h * p.T + t.lo + key] = NAN;
    }
    if (GROUPED && t.sums) store_row<DK>(t.sums, t.lo * ldk + t.hk * DK, ldk, rows, kB, key, l >> 4, dk, 0);
    else store_row<DK>(p.dk_out, t.lo * ldk + t.hk * DK, ldk, rows, kB, key, l >> 4, dk, p.out_bf16);
}

template <typename T, int DK, int DV, bool GROUPED>
__device__ __forceinline__ void dv_role(const LinearBwdParams& p, const Task& t, GradTiles<T, DK, DV>& s) {
    typedef typename V8<T>::t frag;
    constexpr int RK = 16 * DK * sizeof(T), RV = 16 * DV * sizeof(T);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rb = row_block(w), rows = t.rows;
    const int64_t ldk = (int64_t)p.Hk * DK, ldv = (int64_t)p.H * DV;

    for (int h = t.h0; h < (GROUPED ? t.h1 : t.h0 + 1); ++h) {
        const bool first = !GROUPED || h == t.h0;
        const int tid = GROUPED ? opaque(threadIdx.x) : threadIdx.x, l = tid & 63, cl = l & 15, qg = l >> 4, key = 16 * rb + cl;
        // the keys in the k order of the state's columns as they are read here
        frag kf[DK / 32];
        row_perms<T, DK>(kf, (const T*)p.k + t.lo * ldk + t.hk * DK, ldk, key, rows, qg);
        Tile<T, kB, DV, kGradThreads> to;
        to.load((const T*)p.dO + t.lo * ldv + h * DV, ldv, rows, tid);
        {
            Tile<T, DK, DV, kGradThreads> td, ts;
            td.load((const T*)p.dS + (t.slot * p.H + h) * DK * DV, DV, DK, tid);
            ts.load((const T*)p.S + (t.slot * p.H + h) * DK * DV, DV, DK, tid);
            Tile<T, kB, DK, kGradThreads> tq;
            if (first) tq.load((const T*)p.q + t.lo * ldk + t.hk * DK, ldk, rows, tid);
            if (w == 0) block_gates(s.G, p.g + (p.g_stride ? t.lo * p.g_stride : 0) + h, p.g_stride, rows, l);
            td.store(s.b, tid);
            float cross = 0.f;
#pragma unroll
            for (int i = 0; i < Tile<T, DK, DV, kGradThreads>::PIECES; ++i) {
                typedef T piece __attribute__((ext_vector_type(16 / sizeof(T))));
                const piece x = __builtin_bit_cast(piece, ts.r[i]), y = __builtin_bit_cast(piece, td.r[i]);
#pragma unroll
                for (int j = 0; j < (int)(16 / sizeof(T)); ++j) cross += to_f32(x[j]) * to_f32(y[j]);
            }
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) cross += __shfl_xor(cross, m, 64);
            if (l == 0) s.sum[w] = cross;
            if (first) tq.store(s.a, tid);
        }
        lds_barrier();
        if (tid == 0) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x += s.sum[i];
            p.cross[t.slot * p.H + h] = x * fast_exp2((float)s.G[kB - 1]);
        }
        // through the state's gradient; row = value channel, column = key
        const Lane<T, DK> lk(cl, qg);
        const Lane<T, DV> lv(cl, qg);
        const double gk = s.G[key];
        const float wj = fast_exp2((float)(s.G[kB - 1] - gk));
        f32x4 dv[DV / 16];
#pragma unroll
        for (int m = 0; m < DV / 16; m += 2) {
            f32x4 x[2] = {zero4(), zero4()};
#pragma unroll
            for (int y = 0; y < DK / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) x[u] = mma_k32(x[u], lv.col(s.b, 2 * y * RV, m + u), kf[y]);
#pragma unroll
            for (int u = 0; u < 2; ++u) dv[m + u] = x[u] * wj;
        }
        lds_barrier();   // the last readers of dS are done
        put_finite(s, to, s.b, tid, w);
        const double gref = s.G[16 * rb + 15];
        const float fk = fast_exp2((float)(gref - gk)) * p.scale;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (l + 64 * i >= 16 * rb + 16) s.F[w][l + 64 * i] = fast_exp2((float)(s.G[l + 64 * i] - gref));
        lds_barrier();
        for (int x = rb / 2; x < (rows + 31) / 32; ++x) {
            f32x4 a[2] = {zero4(), zero4()};
#pragma unroll
            for (int y = 0; y < DK / 32; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) a[u] = mma_k32(a[u], lk.perm(s.a, (2 * x + u) * RK, y), kf[y]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = 2 * x + u;
                if (n > rb) {
                    a[u] *= lds4(&s.F[w][16 * n + 4 * qg]) * fk;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int query = 16 * n + 4 * qg + i;
                        a[u][i] = keep(a[u][i] * (fast_exp2((float)(s.G[query] - gk)) * p.scale), key <= query);
                    }
                }
            }
            const frag f = pack8<T>(a[0], a[1]);   // bf16 inputs: P rounded to the products' type
#pragma unroll
            for (int m = 0; m < DV / 16; ++m) dv[m] = mma_k32(dv[m], lv.col(s.b, 2 * x * RV, m), f);
        }
        if (any_odd(s)) odd_results<T, DV>(dv, (const T*)p.dO + t.lo * ldv + h * DV, ldv, rows, rb / 2, kB / 32, cl, qg, [&](int query) { return key <= query; });
        store_row<DV>(p.dv_out, t.lo * ldv + h * DV, ldv, rows, kB, key, qg, dv, p.out_bf16);
        if constexpr (GROUPED) lds_barrier();   // the last readers of this head's tiles are done
    }
}

// GROUPED: several value heads to a key head.
template <typename T, int DK, int DV, bool GROUPED>
__global__ __launch_bounds__(kGradThreads, sizeof(T) == 2 ? 4 : 2) void linear_grads_kernel(LinearBwdParams p) {
    __shared__ GradTiles<T, DK, DV> s;
    const int64_t group = blockIdx.x / 24;
    const int x = (int)(blockIdx.x % 24), role = x >> 3;
    const int64_t task = group * 8 + (x & 7);
    const int units = GROUPED ? p.Hk * p.parts : p.Hk, unit = (int)(task % units), part = GROUPED ? unit % p.parts : 0;
    Task t;
    t.slot = task / units;
    if (t.slot >= p.blocks) return;
    t.hk = GROUPED ? unit / p.parts : unit;
    const int R = p.H / p.Hk;
    t.h0 = GROUPED ? t.hk * R + part * (R / p.parts) : t.hk;
    t.h1 = GROUPED ? t.h0 + R / p.parts : t.hk + 1;
    t.sums = nullptr;
    if (GROUPED && p.parts > 1) t.sums = p.sums + (int64_t)(role * p.parts + part) * p.T * p.Hk * DK;   // dv has none
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, t.slot, kB);
    t.lo = rg.lo;
    t.rows = (int)(rg.hi - rg.lo);
    if (t.rows <= 0) return;
    if (role == 0) dq_role<T, DK, DV, GROUPED>(p, t, s);
    else if (role == 1) dk_role<T, DK, DV, GROUPED>(p, t, s);
    else dv_role<T, DK, DV, GROUPED>(p, t, s);
}

// dq (blockIdx.y 0) and dk of some rows of a block and key head from the sums of its
// parts, in their order.
template <int DK>
__global__ __launch_bounds__(kThreads) void linear_parts_kernel(LinearBwdParams p) {
    constexpr int LANES = DK / 4, ROWS = kThreads / LANES, PIECES = kB / ROWS;
    const int64_t id = blockIdx.x / PIECES, slot = id / p.Hk;
    const int hk = (int)(id % p.Hk), row = blockIdx.x % PIECES * ROWS + threadIdx.x / LANES;
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, kB);
    if (row >= rg.hi - rg.lo) return;
    const int64_t plane = p.T * p.Hk * DK, at = ((rg.lo + row) * p.Hk + hk) * DK + threadIdx.x % LANES * 4;
    const float* from = p.sums + blockIdx.y * p.parts * plane + at;
    f32x4 sum = lds4(from);
#pragma unroll 4
    for (int i = 1; i < p.parts; ++i) sum += lds4(from + i * plane);
    store4(blockIdx.y ? p.dk_out : p.dq, at, sum, p.out_bf16);
}

// dg of a block and 32 heads, two of them a wave: lane l holds tokens l and l + 64.  64-bit sums.
// They leave through LDS, a token's heads together: single ones, a row apart each, took 13 us
// at 32768 tokens x 32 heads, this 10.
constexpr int kDgHeads = 32;
__global__ __launch_bounds__(1024) void linear_dg_kernel(LinearBwdParams p) {
    __shared__ float out[kB][kDgHeads + 1];
    const int tid = threadIdx.x, l = tid & 63, groups = (p.H + kDgHeads - 1) / kDgHeads;
    const int64_t slot = blockIdx.x / groups;
    const int h0 = (int)(blockIdx.x % groups) * kDgHeads;
    const Range rg = piece_range(p.cu, p.N, p.seqlen, p.T, slot, kB);
    const int rows = (int)(rg.hi - rg.lo);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int hu = (tid >> 6) + 16 * u, h = h0 + hu;
        if (h >= p.H) break;
        const int64_t id = slot * p.H + h, at = (int64_t)h * p.T + rg.lo;
        if (rows <= 0) {
            if (p.dg_part && l == 0) p.dg_part[id] = 0.f;
            continue;
        }
        double x[2], f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = l + 64 * i;
            x[i] = t < rows ? (double)p.e[at + t] - (double)p.a[at + t] : 0.0;
            f[i] = t < rows ? (double)p.f[at + t] : 0.0;
        }
        const double c = p.cross[id];
        double xs[2], fs[2];
        xs[0] = wave_scan(x[0]);
        fs[0] = wave_scan(f[0]);
        xs[1] = wave_scan(x[1]) + last_lane(xs[0]);
        fs[1] = wave_scan(f[1]) + last_lane(fs[0]);
        const double all = last_lane(xs[1]);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = l + 64 * i;
            const double d = (all - xs[i] + x[i]) + (fs[i] - f[i]) + c;
            if (t < rows) sum += d;
            out[t][hu] = (float)d;
        }
        if (p.dg_part) {
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, 64);
            if (l == 0) p.dg_part[id] = (float)sum;
        }
    }
    if (p.dg_part) return;
    __syncthreads();
    const int h = h0 + tid % kDgHeads;
    if (h < p.H)
        for (int t = tid / kDgHeads; t < rows; t += 1024 / kDgHeads) store1(p.dg, (rg.lo + t) * p.H + h, out[t][tid % kDgHeads], p.dg_bf16);
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
    if (tid == 0) store1(p.dg, h, (float)s[0], p.dg_bf16);
}

template <typename T, int DK, int DV> static void grads_t(const LinearBwdParams& p, hipStream_t stream) {
    const int64_t tasks = (p.blocks * p.Hk * p.parts + 7) / 8 * 8;
    const dim3 grid((unsigned)(tasks * 3));
    if (p.H == p.Hk) hipLaunchKernelGGL((linear_grads_kernel<T, DK, DV, false>), grid, dim3(kGradThreads), 0, stream, p);
    else hipLaunchKernelGGL((linear_grads_kernel<T, DK, DV, true>), grid, dim3(kGradThreads), 0, stream, p);
    if (p.parts > 1) hipLaunchKernelGGL(linear_parts_kernel<DK>, dim3((unsigned)(p.blocks * p.Hk * (kB * DK / (4 * kThreads))), 2), dim3(kThreads), 0, stream, p);
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
        hipLaunchKernelGGL(linear_dg_kernel, dim3((unsigned)(p.blocks * ((p.H + kDgHeads - 1) / kDgHeads))), dim3(1024), 0, stream, p);
    }
    if (p.dg_part) hipLaunchKernelGGL(linear_dg_head_kernel, dim3(p.H), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace kda
