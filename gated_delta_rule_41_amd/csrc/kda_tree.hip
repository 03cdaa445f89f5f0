// kda_tree.hip -- a tree of drafted tokens over a recurrent state.
//
// Speculative decoding drafts a tree of tokens on top of a sequence's state S.  Node i sees
// the state after its own path root .. i, so with G_i the sum of its path's gates (per key
// channel for the delta rule, per head for the linear rule) and a running over i's ancestors:
//   delta:   u_i = beta_i (v_i - S^T (kh_i e^{G_i})) - beta_i sum_a (kh_i . kh_a e^{G_i-G_a}) u_a
//            o_i = S^T (qh_i e^{G_i}) + sum_{a or i} (qh_i . kh_a e^{G_i-G_a}) u_a
//   linear:  o_i = scale (e^{G_i} S^T q_i + sum_{a or i} (q_i . k_a) e^{G_i-G_a} v_a)
// which reads the state once for all nodes and never forms a node's state.  The decay
// between a node and an ancestor is the product of the factors e^g passed on the way up
// (each at most 1, so any g <= 0 works), and only true ancestor pairs are visited.
//
// kda_tree_kernel: one workgroup per (sequence, head), every load issued first.  16 lanes per
// node climb its path (A matrices, e^{G_i}) while the state arrives; one matrix product of all
// rows with the state, transposed, so that a wave keeps its 16 value columns of every node and
// solves for them alone: level by level from the roots, every deeper node takes what its
// ancestor of that level adds to u and o, one read of u for both.  Sums run over true ancestors
// only, so nothing in another branch, NaN included, reaches a node.
//
// 64 trees of 61 nodes x 32 heads of 128, bf16, delta rule: 91 to 97 us, 0.29 GB at 3.1 TB/s; vector
// instructions issue 71% of the time, two workgroups a compute unit in turn through load (a third
// of a workgroup's time), climb, products, solve.  One workgroup with the solve level by level
// across waves took 247 us, two 119, each wave for itself 100.  Linear rule, 32 nodes: 43.0 us,
// 4.1 TB/s.  fp32 inputs: 186 us at 128 x 128, where one workgroup fits a compute unit, 67 at 64 x 64,
// the linear rule 52.
//
// kda_tree_commit_kernel: the recurrence along the accepted path with the state in registers,
// read and written once (kda_decode's layout).  128 sequences x 32 heads, paths of up to 7 nodes:
// 110 us, 5.1 TB/s, a copy's rate.
#include "kda_linear_device.h"
#include "kda_tree.h"

namespace kda {
using namespace lin;

typedef unsigned long long u64;

// The parent of node a of a tree: -1 for the state, below -1 if the node is absent (its entry
// is below -1, or is not smaller than its own index).  `par` is an LDS array of 64.
__device__ __forceinline__ int parent_of(const int* par, int a, int L) {
    const int up = a < L ? par[a] : -2;
    return up < a ? up : -2;
}

__device__ __forceinline__ float sigmoidf(float b) { return 1.f / (1.f + __expf(-b)); }

// 1 / sqrt(x) by the hardware's instruction, which is off by a unit in the last place at most but
// takes x below fp32's smallest normal number for zero: such sums are scaled up first.  (Division
// and square root as the compiler makes them: 64 trees of 61 nodes x 32 heads 98.1 us, this 97.1.)
__device__ __forceinline__ float inv_sqrt(float x) {
    const bool tiny = x < 0x1p-100f;
    return __builtin_amdgcn_rsqf(tiny ? x * 0x1p96f : x) * (tiny ? 0x1p48f : 1.f);
}

// Eight elements of a global row as fp32.
template <typename T> __device__ __forceinline__ f32x8 load8f(const T* p) {
    return widen8(*reinterpret_cast<const typename V8<T>::t*>(p));
}
__device__ __forceinline__ float dot8(f32x8 a, f32x8 b) {
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) x += a[j] * b[j];
    return x;
}
__device__ __forceinline__ f32x8 splat8(float x) { return f32x8{x, x, x, x, x, x, x, x}; }

// An fp32 operand with fp32 accuracy in a product with another: bf16 inputs take two bf16 terms
// each and three products (the fourth is below 2^-16 of the result), fp32 inputs the fp32 unit.
template <typename T> struct Two;
template <> struct Two<bf16> {
    static constexpr int PLANES = 2;
    bf16x8 h, l;
    // bf16's largest value in the first term where x is larger or infinite: what is left is x's then
    __device__ __forceinline__ void set(f32x8 x) {
        f32x8 y;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __builtin_amdgcn_fmed3f(x[j], -0x1.fep127f, 0x1.fep127f);
        h = __builtin_convertvector(y, bf16x8);
        l = __builtin_convertvector(x - widen8(h), bf16x8);
    }
    template <int COLS> __device__ __forceinline__ void get(const Lane<bf16, COLS>& at, const bf16* t, int plane, int off, int y) {
        h = at.row(t, off, y);
        l = at.row(t + plane, off, y);
    }
};
template <> struct Two<float> {
    static constexpr int PLANES = 1;
    f32x8 h;
    __device__ __forceinline__ void set(f32x8 x) { h = x; }
    template <int COLS> __device__ __forceinline__ void get(const Lane<float, COLS>& at, const float* t, int, int off, int y) { h = at.row(t, off, y); }
};
__device__ __forceinline__ f32x4 mma_two(f32x4 c, const Two<bf16>& a, const Two<bf16>& b) {
    c = mma_k32(c, a.l, b.h);
    c = mma_k32(c, a.h, b.l);
    return mma_k32(c, a.h, b.h);
}
__device__ __forceinline__ f32x4 mma_two(f32x4 c, const Two<float>& a, const Two<float>& b) { return mma_k32(c, a.h, b.h); }

// A lane's E channels (8 or 4, at E cl) of a row in LDS.
template <typename T, int E> __device__ __forceinline__ f32x8 get_row(const T* row, int cl) {
    if constexpr (E == 4) {
        const f32x4 x = unpack4(lds4(row + 4 * cl));
        return f32x8{x[0], x[1], x[2], x[3], 0.f, 0.f, 0.f, 0.f};
    } else if constexpr (sizeof(T) == 2) {
        return widen8(*reinterpret_cast<const bf16x8*>(row + 8 * cl));
    } else {   // fp32: the halves of all lanes apart, 16 bytes a lane each, for conflict-free reads
        return join(lds4(row + 4 * cl), lds4(row + 64 + 4 * cl));
    }
}
template <int E> __device__ __forceinline__ void put_row(float* row, int cl, f32x8 x) {
    *reinterpret_cast<f32x4*>(row + 4 * cl) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
    if constexpr (E == 8) *reinterpret_cast<f32x4*>(row + 64 + 4 * cl) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
}
template <int E> __device__ __forceinline__ void put_row(bf16* row, int cl, f32x8 x) {   // exact: the values were bf16
    const bf16x8 y = __builtin_convertvector(x, bf16x8);
    if constexpr (E == 8) *reinterpret_cast<bf16x8*>(row + 8 * cl) = y;
    else *reinterpret_cast<bf16x4*>(row + 4 * cl) = __builtin_shufflevector(y, y, 0, 1, 2, 3);
}
// The same channels of an operand tile (Swz), in planes.
template <int E, int DK> __device__ __forceinline__ void put_planes(float* t, int, int row, int cl, f32x8 x) {
    typedef Swz<float, DK> Z;
    const f32x4 lo = __builtin_shufflevector(x, x, 0, 1, 2, 3), hi = __builtin_shufflevector(x, x, 4, 5, 6, 7);
    *reinterpret_cast<f32x4*>(t + Z::at(row, E == 8 ? 2 * cl : cl)) = lo;
    if constexpr (E == 8) *reinterpret_cast<f32x4*>(t + Z::at(row, 2 * cl + 1)) = hi;
}
template <int E, int DK> __device__ __forceinline__ void put_planes(bf16* t, int plane, int row, int cl, f32x8 x) {
    typedef Swz<bf16, DK> Z;
    Two<bf16> y;
    y.set(x);
    if constexpr (E == 8) {
        *reinterpret_cast<bf16x8*>(t + Z::at(row, cl)) = y.h;
        *reinterpret_cast<bf16x8*>(t + plane + Z::at(row, cl)) = y.l;
    } else {
        const int o = Z::at(row, cl >> 1) + 4 * (cl & 1);
        *reinterpret_cast<bf16x4*>(t + o) = __builtin_shufflevector(y.h, y.h, 0, 1, 2, 3);
        *reinterpret_cast<bf16x4*>(t + plane + o) = __builtin_shufflevector(y.l, y.l, 0, 1, 2, 3);
    }
}

// LDS of a tree of up to NL nodes.  The first part is, one after the other: the keys and e^g
// (climb), the rows that meet the state, u.
template <typename T, bool DELTA, int NL, int DK, int DV> struct TreeShared {
    static constexpr int LU = DV + 4, PLANE = NL * DK;
    struct Climb {
        T k[NL * DK];
        float a[DELTA ? NL * DK : NL];
    };
    union {
        __align__(32) char bytes[1];
        Climb c;
        T rows[Two<T>::PLANES * PLANE];
        float u[NL * LU];
    } x;
    // node i's path and its products with it: entry i (i + 1) / 2 + d for the node d steps up.
    // Entry 0 is node i itself with products of zero, where a node waits once its path is used up.
    static constexpr int ENTRIES = NL * (NL + 1) / 2;
    float kk[DELTA ? ENTRIES : 1], qk[ENTRIES];
    unsigned char node[ENTRIES];
    float self[NL], beta[NL], norm[NL];   // self: q_i . k_i
    int par[64], depth[NL];               // depth: strict ancestors, -1 of an absent node
};

// NL: the tree's size rounded up to 16, 32 or 64 nodes.
template <typename T, bool DELTA, int NL, int DK, int DV>
__global__ __launch_bounds__(NL == 16 ? 256 : 512, sizeof(T) == 2 ? 4 : 2) void kda_tree_kernel(TreeParams p) {
    constexpr int THREADS = NL == 16 ? 256 : 512, WAVES = THREADS / 64, E = DK / 16, CG = DV / 16, MT = NL / 16;
    constexpr int NODES = THREADS / 16, ROUNDS = NL / NODES;   // nodes that climb at once
    // column groups: COLS a wave, or shared by STEP waves that take every STEP-th tile of nodes
    constexpr int STEP = WAVES > CG ? WAVES / CG : 1, COLS = WAVES < CG ? CG / WAVES : 1;
    typedef TreeShared<T, DELTA, NL, DK, DV> Shared;
    __shared__ __align__(32) Shared s;

    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63, cl = l & 15, qg = l >> 4;
    const int64_t nh = blockIdx.x, n = nh / p.H;
    const int h = (int)(nh % p.H), hk = h / (p.H / p.Hk), L = p.L;
    const int64_t node0 = n * L;

    if (tid < 64) s.par[tid] = tid < L ? p.parent[node0 + tid] : -2;
    f32x8 kv[ROUNDS], qv[ROUNDS], av[ROUNDS];
    float bt[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int i = (tid >> 4) + r * NODES;
        const int64_t at = node0 + (i < L ? i : 0);
        const T* kp = (const T*)p.k + (at * p.Hk + hk) * DK + E * cl;
        const T* qp = (const T*)p.q + (at * p.Hk + hk) * DK + E * cl;
        if constexpr (E == 8) {
            kv[r] = load8f(kp);
            qv[r] = load8f(qp);
        } else {
            const f32x4 a = unpack4(*reinterpret_cast<const typename V4<T>::t*>(kp)), b = unpack4(*reinterpret_cast<const typename V4<T>::t*>(qp));
            kv[r] = f32x8{a[0], a[1], a[2], a[3], 0.f, 0.f, 0.f, 0.f};
            qv[r] = f32x8{b[0], b[1], b[2], b[3], 0.f, 0.f, 0.f, 0.f};
        }
        bt[r] = 0.f;
        if constexpr (DELTA) {
            const T* gp = (const T*)p.g + (at * p.H + h) * DK + E * cl;
            f32x8 g = splat8(0.f);
            if constexpr (E == 8) g = load8f(gp);
            else {
                const f32x4 a = unpack4(*reinterpret_cast<const typename V4<T>::t*>(gp));
                g = f32x8{a[0], a[1], a[2], a[3], 0.f, 0.f, 0.f, 0.f};
            }
            av[r] = g;
            bt[r] = to_f32(((const T*)p.beta)[at * p.H + h]);
        } else {
            av[r] = splat8(((const float*)p.g)[p.gate_head ? h : at * p.H + h]);
        }
    }
    // the state as product fragments: value column 16 cg + cl, rows 32 y + 8 qg + j
    Two<T> st[COLS][DK / 32];
    {
        f32x8 x[COLS][DK / 32];
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const float* sp = p.s_in + nh * DK * DV + 16 * (w % CG + c * WAVES) + cl;
#pragma unroll
            for (int y = 0; y < DK / 32; ++y)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[c][y][j] = p.s_in ? sp[(32 * y + 8 * qg + j) * DV] : 0.f;
        }
        // norms, gates and the keys' rows meanwhile
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int i = (tid >> 4) + r * NODES;
            put_row<E>(s.x.c.k + i * DK, cl, kv[r]);
            if constexpr (DELTA) {
                const float rk = inv_sqrt(row16_sum(dot8(kv[r], kv[r])) + p.eps);
                const float rq = p.scale * inv_sqrt(row16_sum(dot8(qv[r], qv[r])) + p.eps);
                kv[r] *= splat8(rk);
                qv[r] *= splat8(rq);
#pragma unroll
                for (int j = 0; j < E; ++j) av[r][j] = fast_exp(av[r][j]);
                put_row<E>(s.x.c.a + i * DK, cl, av[r]);
                if (cl == 0) {
                    s.norm[i] = rk;
                    s.beta[i] = sigmoidf(bt[r]);
                }
            } else {
                qv[r] *= splat8(p.scale);
                av[r] = splat8(fast_exp(av[r][0]));
                if (cl == 0) s.x.c.a[i] = av[r][0];
            }
        }
        __syncthreads();
        // climb: node i's products with its path, and the product of the factors passed
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int i = (tid >> 4) + r * NODES;
            const int t0 = i * (i + 1) / 2;
            const float self = row16_sum(dot8(qv[r], kv[r]));
            if (cl == 0) {
                s.self[i] = self;
                s.node[t0] = (unsigned char)i;
                s.qk[t0] = 0.f;
                if constexpr (DELTA) s.kk[t0] = 0.f;
            }
            int d = 0, a = parent_of(s.par, i, L);
            for (; a >= 0; a = parent_of(s.par, a, L)) {
                const f32x8 ke = get_row<T, E>(s.x.c.k + a * DK, cl) * av[r];
                float norm = 1.f;
                if constexpr (DELTA) {
                    norm = s.norm[a];
                    av[r] *= get_row<float, E>(s.x.c.a + a * DK, cl);
                } else {
                    av[r] *= splat8(s.x.c.a[a]);
                }
                ++d;
                const float qk = row16_sum(dot8(qv[r], ke)) * norm;
                if constexpr (DELTA) {
                    const float kk = row16_sum(dot8(kv[r], ke)) * norm;
                    if (cl == 0) s.kk[t0 + d] = kk;
                }
                if (cl == 0) {
                    s.qk[t0 + d] = qk;
                    s.node[t0 + d] = (unsigned char)a;
                }
            }
            if (cl == 0) s.depth[i] = a < -1 ? -1 : d;
        }
#pragma unroll
        for (int c = 0; c < COLS; ++c)
#pragma unroll
            for (int y = 0; y < DK / 32; ++y) st[c][y].set(x[c][y]);
    }

    // v meanwhile; value columns 16 cg + 4 qg + i of node 16 m + cl, as the products below
    auto mine = [&](int m) { return STEP == 1 || m % STEP == w / CG; };
    auto column = [&](int c) { return 16 * (w % CG + c * WAVES) + 4 * qg; };
    typename V4<T>::t v[COLS][MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = 16 * m + cl < L ? 16 * m + cl : 0;
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            if (mine(m)) v[c][m] = *reinterpret_cast<const typename V4<T>::t*>((const T*)p.v + ((node0 + i) * p.H + h) * DV + column(c));
    }
    // rows times the state; row = value column 16 cg + 4 qg + i, column = node 16 m + cl
    const Lane<T, DK> lane(cl, qg);
    constexpr int R16 = 16 * DK * sizeof(T);
    f32x4 ks[COLS][MT], qs[COLS][MT];
#pragma unroll
    for (int pass = DELTA ? 0 : 1; pass < 2; ++pass) {
        __syncthreads();   // the last readers of this part of LDS are done
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            put_planes<E, DK>(s.x.rows, Shared::PLANE, (tid >> 4) + r * NODES, cl, (pass ? qv[r] : kv[r]) * av[r]);
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            f32x4 x[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) x[c] = zero4();
            if (mine(m) && 16 * m < L) {
#pragma unroll
                for (int y = 0; y < DK / 32; ++y) {
                    Two<T> f;
                    f.get(lane, s.x.rows, Shared::PLANE, m * R16, y);
#pragma unroll
                    for (int c = 0; c < COLS; ++c) x[c] = mma_two(x[c], st[c][y], f);
                }
            }
#pragma unroll
            for (int c = 0; c < COLS; ++c) (pass ? qs : ks)[c][m] = x[c];
        }
    }
    __syncthreads();
    // Nodes of depth 0, 1, ...: their u is complete, and every deeper node takes its part of
    // u and o from its ancestor of that depth.  A wave needs no other wave's columns, and a
    // wave's LDS operations are done in order; only where waves share columns (STEP) they wait
    // for each other.
    int depth[MT], at[MT], a[MT], levels = 0;   // at: the entry of the next ancestor, a
    float beta[MT], self[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = 16 * m + cl;
        depth[m] = s.depth[i];
        at[m] = i * (i + 1) / 2 + (depth[m] > 0 ? depth[m] : 0);
        a[m] = s.node[at[m]];
        beta[m] = DELTA ? s.beta[i] : 1.f;
        self[m] = s.self[i];
        while (__ballot(depth[m] >= levels)) ++levels;
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            if (mine(m)) ks[c][m] = DELTA ? unpack4(v[c][m]) - ks[c][m] : unpack4(v[c][m]);
    }
    for (int d = 0; d < levels; ++d) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (mine(m) && depth[m] == d) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const f32x4 u = beta[m] * ks[c][m];
                    qs[c][m] += self[m] * u;
                    *reinterpret_cast<f32x4*>(s.x.u + (16 * m + cl) * Shared::LU + column(c)) = u;
                }
            }
        if (d + 1 == levels) break;
        if constexpr (STEP > 1) __syncthreads();
        else asm volatile("" ::: "memory");
        // without branches, so that the reads of all nodes are in flight together; a node whose
        // path is used up adds zero times its own u
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if (mine(m)) {
                float kk = 0.f;
                if constexpr (DELTA) kk = s.kk[at[m]];
                const float qk = s.qk[at[m]];
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const f32x4 u = *reinterpret_cast<const f32x4*>(s.x.u + a[m] * Shared::LU + column(c));
                    if constexpr (DELTA) ks[c][m] -= kk * u;
                    qs[c][m] += qk * u;
                }
                at[m] -= depth[m] > d;
                a[m] = s.node[at[m]];
            }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = 16 * m + cl;
        if (mine(m) && i < L) {
#pragma unroll
            for (int c = 0; c < COLS; ++c)
                store4(p.o, ((node0 + i) * p.H + h) * DV + column(c), depth[m] >= 0 ? qs[c][m] : zero4(), p.out_bf16);
        }
    }
}

template <typename T, bool DELTA, int DK>
__global__ __launch_bounds__(kThreads) void kda_tree_commit_kernel(TreeParams p) {
    constexpr int RPT = DK / 16, BATCH = 8;
    __shared__ float sk[BATCH][DK], sal[BATCH][DK], sb[BATCH];
    __shared__ f32x4 sred[2][4][16];
    __shared__ int sPar[64];
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, tc = tid & 15, tr = tid >> 4;
    const int slices = p.dv / kSlice;
    const int64_t nh = blockIdx.x / slices, n = nh / p.H;
    const int slice = blockIdx.x % slices, h = (int)(nh % p.H), hk = h / (p.H / p.Hk);
    const int col = slice * kSlice + 4 * tc;
    const int64_t base = nh * DK * p.dv + col, node0 = n * p.L;

    f32x4 s[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j)
        s[j] = p.s_in ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p.s_in + base + (int64_t)(tr + 16 * j) * p.dv)) : zero4();
    if (tid < 64) sPar[tid] = tid < p.L ? p.parent[node0 + tid] : -2;
    const int leaf = p.accept[n];
    __syncthreads();
    // the path as a bit mask: a parent's index is below its child's, so ascending bits run from the root
    u64 path = 0;
    if (leaf >= 0 && leaf < p.L) {
        int a = leaf;
        for (; a >= 0; a = parent_of(sPar, a, p.L)) path |= 1ull << a;
        if (a < -1) path = 0;   // an absent node
    }
    for (int done = 0; path;) {
        const int count = __popcll(path) < BATCH ? __popcll(path) : BATCH;
        // 32 lanes per node: kh, e^g, beta of up to BATCH nodes
        {
            const int b = tid >> 5, c = tid & 31;
            u64 m = path;
            for (int x = 0; x < b; ++x) m &= m - 1;
            const bool on = b < count;
            const int64_t at = node0 + (on ? __ffsll((long long)m) - 1 : 0);
            float kx[DK / 32], sum = 0.f;
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                kx[e] = to_f32(((const T*)p.k)[(at * p.Hk + hk) * DK + c + 32 * e]);
                sum += kx[e] * kx[e];
            }
            float r = 1.f;
            if constexpr (DELTA) {
#pragma unroll
                for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor(sum, x, 64);
                r = inv_sqrt(sum + p.eps);
            }
            if (done) __syncthreads();   // the last batch's readers are done
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                sk[b][c + 32 * e] = kx[e] * r;
                if constexpr (DELTA)
                    sal[b][c + 32 * e] = fast_exp(to_f32(((const T*)p.g)[(at * p.H + h) * DK + c + 32 * e]));
            }
            if (c == 0) {
                if constexpr (DELTA) sb[b] = sigmoidf(to_f32(((const T*)p.beta)[at * p.H + h]));
                else sb[b] = fast_exp(((const float*)p.g)[p.gate_head ? h : at * p.H + h]);
            }
        }
        __syncthreads();
        for (int b = 0; b < count; ++b) {
            const int64_t at = node0 + __ffsll((long long)path) - 1;
            path &= path - 1;
            f32x4 u = unpack4(*reinterpret_cast<const typename V4<T>::t*>((const T*)p.v + (at * p.H + h) * p.dv + col));
            if constexpr (DELTA) {
                f32x4 x = zero4();
#pragma unroll
                for (int j = 0; j < RPT; ++j) {
                    s[j] *= sal[b][tr + 16 * j];
                    x += sk[b][tr + 16 * j] * s[j];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] += __shfl_xor(x[e], 16, 64);
                    x[e] += __shfl_xor(x[e], 32, 64);
                }
                if (l < 16) sred[b & 1][w][tc] = x;
                __syncthreads();
                x = (sred[b & 1][0][tc] + sred[b & 1][1][tc]) + (sred[b & 1][2][tc] + sred[b & 1][3][tc]);
                u = sb[b] * (u - x);
            }
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                if constexpr (!DELTA) s[j] *= sb[b];
                s[j] += sk[b][tr + 16 * j] * u;
            }
        }
        done += count;
    }
#pragma unroll
    for (int j = 0; j < RPT; ++j)
        __builtin_nontemporal_store(s[j], reinterpret_cast<f32x4*>(p.s_out + base + (int64_t)(tr + 16 * j) * p.dv));
}

template <typename T, bool DELTA, int NL, int DK> static void tree_n(const TreeParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.N * p.H));
    if (p.dv == 128) hipLaunchKernelGGL((kda_tree_kernel<T, DELTA, NL, DK, 128>), grid, dim3(NL == 16 ? 256 : 512), 0, stream, p);
    else hipLaunchKernelGGL((kda_tree_kernel<T, DELTA, NL, DK, 64>), grid, dim3(NL == 16 ? 256 : 512), 0, stream, p);
}
template <typename T, bool DELTA, int DK> static void tree_t(const TreeParams& p, hipStream_t stream) {
    if (p.L <= 16) tree_n<T, DELTA, 16, DK>(p, stream);
    else if (p.L <= 32) tree_n<T, DELTA, 32, DK>(p, stream);
    else tree_n<T, DELTA, 64, DK>(p, stream);
}
template <typename T, bool DELTA, int DK> static void commit_t(const TreeParams& p, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.N * p.H * (p.dv / kSlice)));
    hipLaunchKernelGGL((kda_tree_commit_kernel<T, DELTA, DK>), grid, dim3(kThreads), 0, stream, p);
}
#define KDA_TREE_DISPATCH(F)                                                                 \
    if (p.N == 0) return hipSuccess;                                                         \
    if (in_dtype == 1) {                                                                     \
        if (delta) dk == 128 ? F<bf16, true, 128>(p, stream) : F<bf16, true, 64>(p, stream); \
        else dk == 128 ? F<bf16, false, 128>(p, stream) : F<bf16, false, 64>(p, stream);     \
    } else {                                                                                 \
        if (delta) dk == 128 ? F<float, true, 128>(p, stream) : F<float, true, 64>(p, stream); \
        else dk == 128 ? F<float, false, 128>(p, stream) : F<float, false, 64>(p, stream);   \
    }                                                                                        \
    return hipGetLastError();

hipError_t launch_tree(const TreeParams& p, bool delta, int in_dtype, int dk, hipStream_t stream) {
    KDA_TREE_DISPATCH(tree_t)
}
hipError_t launch_tree_commit(const TreeParams& p, bool delta, int in_dtype, int dk, hipStream_t stream) {
    KDA_TREE_DISPATCH(commit_t)
}

}  // namespace kda
