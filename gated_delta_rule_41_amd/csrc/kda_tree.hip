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
// kda_tree_kernel: one workgroup per (sequence, head).  The state's loads are issued first
// and are in flight while 16 lanes per node climb its path (A matrices, e^{G_i}); then one
// matrix product of all rows with the state, then the triangular solve level by level of the
// tree (nodes of one depth are independent), then the outputs.
//
// kda_tree_commit_kernel: the recurrence along the accepted path with the state in registers,
// read and written once (kda_decode's layout).
#include "kda_linear_device.h"
#include "kda_tree.h"

namespace kda {
using namespace lin;

typedef unsigned long long u64;

// Lane i of the calling wave takes node i: its strict ancestors as a bit mask and its depth,
// depth -1 for an absent node.  A node is absent if its parent entry is below -1, is not
// smaller than its own index, or names an absent node.  `par` is an LDS array of 64.
__device__ __forceinline__ void climb(const int* par, int i, int L, u64& anc, int& depth) {
    anc = 0;
    depth = 0;
    int a = i;
    while (true) {
        const int up = a < L ? par[a] : -2;
        if (up < -1 || up >= a) {
            depth = -1;
            return;
        }
        if (up == -1) return;
        anc |= 1ull << up;
        ++depth;
        a = up;
    }
}

__device__ __forceinline__ float sigmoidf(float b) { return 1.f / (1.f + __expf(-b)); }

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

// Eight elements of an LDS row (16-byte aligned).
__device__ __forceinline__ f32x8 row8(const float* p) {
    return __builtin_shufflevector(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4), 0, 1, 2, 3, 4, 5, 6, 7);
}

// a * b in fp32 accuracy for bf16 inputs: both fp32 operands as two bf16 terms, three
// products (the fourth is below 2^-16 of the result); fp32 inputs take the fp32 unit.
template <typename T> __device__ __forceinline__ f32x4 mma_split(f32x4 c, f32x8 a, f32x8 b) {
    if constexpr (sizeof(T) == 4) return mma_k32(c, a, b);
    else {
        const bf16x8 ah = __builtin_convertvector(a, bf16x8), bh = __builtin_convertvector(b, bf16x8);
        const bf16x8 al = __builtin_convertvector(a - widen8(ah), bf16x8);
        const bf16x8 bl = __builtin_convertvector(b - widen8(bh), bf16x8);
        c = mma_k32(c, al, bh);
        c = mma_k32(c, ah, bl);
        return mma_k32(c, ah, bh);
    }
}

// NL: the tree's size rounded up to 16, 32 or 64 nodes.
template <typename T, bool DELTA, int NL, int DK, int DV>
__global__ __launch_bounds__(NL * 16) void kda_tree_kernel(TreeParams p) {
    constexpr int THREADS = NL * 16, WAVES = THREADS / 64, LK = DK + 4, LU = DV + 4, E = DK / 16, CG = DV / 16;
    constexpr int ROWS = NL * (LK > LU ? LK : LU);
    __shared__ __align__(32) float sK[ROWS];   // kh, then kh e^G, then u
    __shared__ __align__(32) float sQ[ROWS];   // qh e^G, then S^T (qh e^G)
    __shared__ __align__(32) float sA[DELTA ? NL * LK : NL];   // e^g
    __shared__ float sKK[DELTA ? NL * (NL + 1) : 1], sQK[NL * (NL + 1)];
    __shared__ float sB[NL];
    __shared__ int sPar[64], sDepth[64];
    __shared__ u64 sAnc[64], sLevel[64];
    __shared__ int sLevels;

    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, cl = l & 15, qg = l >> 4;
    const int64_t nh = blockIdx.x, n = nh / p.H;
    const int h = (int)(nh % p.H), hk = h / (p.H / p.Hk), L = p.L, dv = DV;
    const int64_t node0 = n * L;

    // the state as product fragments: column 16 cg + cl, rows 32 s + 8 qg + j.  Waves share the
    // columns' groups; the waves beyond the first CG of them take every STEP-th row tile.
    constexpr int STEP = WAVES > CG ? WAVES / CG : 1, COLS = WAVES < CG ? CG / WAVES : 1;
    f32x8 sf[COLS][DK / 32];
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        const float* s = p.s_in + nh * DK * dv + 16 * (w % CG + c * WAVES) + cl;
#pragma unroll
        for (int x = 0; x < DK / 32; ++x)
#pragma unroll
            for (int j = 0; j < 8; ++j) sf[c][x][j] = p.s_in ? s[(int64_t)(32 * x + 8 * qg + j) * dv] : 0.f;
    }
    if (tid < 64) sPar[tid] = tid < L ? p.parent[node0 + tid] : -2;

    // 16 lanes per node, E channels each
    const int i = tid >> 4;
    f32x8 kv = splat8(0.f), qv = splat8(0.f), av = splat8(1.f);
    const bool in = i < L;
    const int64_t at = node0 + (in ? i : 0);
    float bt = 0.f;
    {
        const T* kp = (const T*)p.k + (at * p.Hk + hk) * DK + E * cl;
        const T* qp = (const T*)p.q + (at * p.Hk + hk) * DK + E * cl;
        if constexpr (E == 8) {
            kv = load8f(kp);
            qv = load8f(qp);
        } else {
            const f32x4 a = unpack4(*reinterpret_cast<const typename V4<T>::t*>(kp));
            const f32x4 b = unpack4(*reinterpret_cast<const typename V4<T>::t*>(qp));
#pragma unroll
            for (int j = 0; j < 4; ++j) { kv[j] = a[j]; qv[j] = b[j]; }
        }
        if constexpr (DELTA) {
            const T* gp = (const T*)p.g + (at * p.H + h) * DK + E * cl;
#pragma unroll
            for (int j = 0; j < E; ++j) av[j] = fast_exp2((float)gate_log2(to_f32(gp[j])));
            bt = sigmoidf(to_f32(((const T*)p.beta)[at * p.H + h]));
            const float nk = row16_sum(dot8(kv, kv)), nq = row16_sum(dot8(qv, qv));
            kv *= splat8(1.f / sqrtf(nk + p.eps));
            qv *= splat8(p.scale / sqrtf(nq + p.eps));
        } else {
            const float g = ((const float*)p.g)[p.gate_head ? h : at * p.H + h];
            av = splat8(fast_exp2((float)gate_log2(g)));
            qv *= splat8(p.scale);
        }
        if (!in) { kv = splat8(0.f); qv = splat8(0.f); }
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
        sK[i * LK + E * cl + j] = kv[j];
        if constexpr (DELTA) sA[i * LK + E * cl + j] = av[j];
    }
    if (cl == 0) {
        if constexpr (!DELTA) sA[i] = av[0];
        sB[i] = bt;
    }
    __syncthreads();
    if (w == 0) {
        u64 anc;
        int depth;
        climb(sPar, l, L, anc, depth);
        sAnc[l] = anc;
        sDepth[l] = depth;
        int levels = 0;
        for (; levels < 64; ++levels) {
            const u64 m = __ballot(depth == levels);
            if (!m) break;
            if (l == 0) sLevel[levels] = m;
        }
        if (l == 0) sLevels = levels;
    }
    __syncthreads();

    // climb: A rows of node i and e^{G_i}; av becomes the product of the factors passed
    const bool live = sDepth[i] >= 0;
    if (live) {
        const float self = row16_sum(dot8(qv, kv));
        if (cl == 0) sQK[i * (NL + 1) + i] = self;
        for (int a = sPar[i]; a >= 0; a = sPar[a]) {
            f32x8 ka = splat8(0.f), aa = splat8(1.f);
#pragma unroll
            for (int j = 0; j < E; ++j) ka[j] = sK[a * LK + E * cl + j];
            if constexpr (DELTA) {
#pragma unroll
                for (int j = 0; j < E; ++j) aa[j] = sA[a * LK + E * cl + j];
            } else {
                aa = splat8(sA[a]);
            }
            const f32x8 ke = ka * av;
            const float qk = row16_sum(dot8(qv, ke));
            if (cl == 0) sQK[i * (NL + 1) + a] = qk;
            if constexpr (DELTA) {
                const float kk = row16_sum(dot8(kv, ke));
                if (cl == 0) sKK[i * (NL + 1) + a] = kk;
            }
            av *= aa;
        }
    }
    __syncthreads();   // every climb has read its kh
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if constexpr (DELTA) sK[i * LK + E * cl + j] = kv[j] * av[j];
        sQ[i * LK + E * cl + j] = qv[j] * av[j];
    }
    __syncthreads();

    // rows times the state; accumulators: row = node 16 m + 4 qg + i, column = value column
    constexpr int MT = NL / 16;
    f32x4 ks[COLS][MT], qs[COLS][MT];
#pragma unroll
    for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            ks[c][m] = qs[c][m] = zero4();
            if ((STEP == 1 || (m % STEP) == w / CG) && 16 * m < L) {
#pragma unroll
                for (int x = 0; x < DK / 32; ++x) {
                    const int r = (16 * m + cl) * LK + 32 * x + 8 * qg;
                    qs[c][m] = mma_split<T>(qs[c][m], row8(sQ + r), sf[c][x]);
                    if constexpr (DELTA) ks[c][m] = mma_split<T>(ks[c][m], row8(sK + r), sf[c][x]);
                }
            }
        }
    __syncthreads();   // sK and sQ change their meaning
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
        const int col = 16 * (w % CG + c * WAVES) + cl;
#pragma unroll
        for (int m = 0; m < MT; ++m)
            if ((STEP == 1 || (m % STEP) == w / CG) && 16 * m < L) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 16 * m + 4 * qg + e;
                    const float v = r < L ? to_f32(((const T*)p.v)[((node0 + r) * p.H + h) * dv + col]) : 0.f;
                    sK[r * LU + col] = DELTA ? sB[r] * (v - ks[c][m][e]) : v;
                    sQ[r * LU + col] = qs[c][m][e];
                }
            }
    }
    __syncthreads();

    // u, level by level: a wave takes a node, a lane DV / 64 columns
    constexpr int CPL = DV / 64;
    if constexpr (DELTA) {
        const int levels = sLevels;
        for (int d = 1; d < levels; ++d) {
            u64 nodes = sLevel[d];
            for (int x = 0; nodes; ++x) {
                const int i2 = __ffsll((long long)nodes) - 1;
                nodes &= nodes - 1;
                if (x % WAVES != w) continue;
                float u[CPL] = {};
                for (u64 m = sAnc[i2]; m; m &= m - 1) {
                    const int a = __ffsll((long long)m) - 1;
                    const float A = sKK[i2 * (NL + 1) + a];
#pragma unroll
                    for (int c = 0; c < CPL; ++c) u[c] += A * sK[a * LU + l + 64 * c];
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) sK[i2 * LU + l + 64 * c] -= sB[i2] * u[c];
            }
            __syncthreads();
        }
    }
    for (int i2 = w; i2 < L; i2 += WAVES) {
        const bool on = sDepth[i2] >= 0;
        float o[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) o[c] = on ? sQ[i2 * LU + l + 64 * c] : 0.f;
        if (on)
            for (u64 m = sAnc[i2] | 1ull << i2; m; m &= m - 1) {
                const int a = __ffsll((long long)m) - 1;
                const float A = sQK[i2 * (NL + 1) + a];
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[c] += A * sK[a * LU + l + 64 * c];
            }
#pragma unroll
        for (int c = 0; c < CPL; ++c) store1(p.o, ((node0 + i2) * p.H + h) * dv + l + 64 * c, o[c], p.out_bf16);
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
        int depth;
        climb(sPar, leaf, p.L, path, depth);
        path = depth < 0 ? 0 : path | 1ull << leaf;
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
                r = 1.f / sqrtf(sum + p.eps);
            }
            if (done) __syncthreads();   // the last batch's readers are done
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                sk[b][c + 32 * e] = kx[e] * r;
                if constexpr (DELTA)
                    sal[b][c + 32 * e] = fast_exp2((float)gate_log2(to_f32(((const T*)p.g)[(at * p.H + h) * DK + c + 32 * e])));
            }
            if (c == 0) {
                if constexpr (DELTA) sb[b] = sigmoidf(to_f32(((const T*)p.beta)[at * p.H + h]));
                else sb[b] = fast_exp2((float)gate_log2(((const float*)p.g)[p.gate_head ? h : at * p.H + h]));
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
    if (p.dv == 128) hipLaunchKernelGGL((kda_tree_kernel<T, DELTA, NL, DK, 128>), grid, dim3(NL * 16), 0, stream, p);
    else hipLaunchKernelGGL((kda_tree_kernel<T, DELTA, NL, DK, 64>), grid, dim3(NL * 16), 0, stream, p);
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
