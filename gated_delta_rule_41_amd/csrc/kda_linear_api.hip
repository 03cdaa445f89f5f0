// kda_linear_api.hip -- the C ABI of the linear rule and of the drafted-tree operators
// (include/kda.h).  As in kda_api.hip every argument is checked on the host before any HIP
// call, and nothing is allocated.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "../../include/kda.h"
#include "kda_internal.h"
#include "kda_linear.h"
#include "kda_tree.h"

#define KDA_TRY(x)                       \
    do {                                 \
        kda_status _s = (x);             \
        if (_s != KDA_OK) return _s;     \
    } while (0)

namespace {

using namespace kda;

kda_status fail(kda_status s, const char* fmt, const char* what = "") {
    snprintf(error_text(), kErrorBytes, fmt, what);
    return s;
}
kda_status launched(hipError_t e) {
    return e == hipSuccess ? KDA_OK : fail(KDA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

kda_status ptr(const void* p, const char* name, bool needed) {
    if (!p) return needed ? fail(KDA_ERR_INVALID_ARG, "%s is NULL", name) : KDA_OK;
    if ((uintptr_t)p & 15) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return KDA_OK;
}

bool is_dtype(int32_t t) { return t == KDA_F32 || t == KDA_BF16; }

kda_status check_heads(int32_t H, int32_t Hk, int32_t dk, int32_t dv, int32_t in, int32_t out, int32_t gate, float scale) {
    if (H < 1 || Hk < 1 || H % Hk) return fail(KDA_ERR_INVALID_ARG, "H and Hk must be >= 1 and Hk must divide H%s");
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return fail(KDA_ERR_UNSUPPORTED, "dk and dv must be 64 or 128%s");
    if (!is_dtype(in) || !is_dtype(out)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype%s");
    if (gate != KDA_GATE_TOKEN && gate != KDA_GATE_HEAD) return fail(KDA_ERR_INVALID_ARG, "unknown gate%s");
    if (!isfinite(scale)) return fail(KDA_ERR_INVALID_ARG, "scale must be finite%s");
    return KDA_OK;
}
int32_t gate_of(const kda_linear_config* c) { return c->gate & ~KDA_GATE_GRAD_F32; }
kda_status check_config(const kda_linear_config* c) {
    if (!c) return fail(KDA_ERR_INVALID_ARG, "config is NULL%s");
    return check_heads(c->H, c->Hk, c->dk, c->dv, c->in_dtype, c->out_dtype, gate_of(c), c->scale);
}

// One launch covers at most 2^32 - 1 work-items along x.
bool grid_fits(int64_t workgroups, int threads) {
    return workgroups >= 0 && workgroups <= (int64_t)UINT32_MAX / threads;
}

// ---------------------------------------------------------------- plans
// A walk goes over a whole document; few documents and heads, or one document much longer than
// the others, leave compute units idle.  Then documents are cut into segments of the tokens
// that would give kWalkTarget workgroups equal shares: the segments' own sums, the states
// entering them, the walks from those.  Documents that fit one segment take no part in the
// first two.  The plan depends on the config and the sizes alone, so that the workspace size
// is a host function; cu_seqlens is on the device, so any document may have all the tokens.
// More than kSegDocs documents are walked whole.  Short ones even out by their number, but a long one
// among them does not: one of 131072 tokens x 16 heads with 511 documents of one token takes 1.1 ms
// forward and 3.7 backward, with 512 of them 9.0 and 7.3.
// Equal shares of small streams would be too short: a segment costs its state four moves
// through memory (T H dk dv / L elements over all of them) and a step of its document's carry
// (T / L of them in a row), against 2 L tokens of walking.  The two square roots are where those
// are equal, with factors from these times (us; forward, 128 x 128, L a floor under the share),
// taken at powers of two as the floor is:
//     tokens x heads         128   256   512  1024
//     2048 x 8                35    40    58   130
//     8192 x 8                70    57    65
//     32768 x 4              108   107    87   110
//     32768 x 8, 16 documents     154   124   127
//     32768 x 1              103    73    75   108
//     131072 x 1             211   211   140   136
// Up to two segments, or eight chunks, are walked whole.  For the backward that is as good: 256 tokens
// x 4 heads of 64, fp32, 35 us whole and 42 cut, 512 tokens 45 and 43; 256 x 8 of 128, bf16, 25 and
// 34, 512 tokens 33 and 37.  The forward takes 26 us whole and 27 cut for 256 of the first, 22 and 25 of
// the second, but 49 and 28, 38 and 26 for 512: the eight chunks cost it that much, and spare calls
// so short a workspace.
constexpr int64_t kWholeTokens = 8 * kLinChunk;

struct Plan {
    int32_t seg_len;     // 0: whole documents
    int32_t whole_len;   // see segment_length
    int64_t chains;      // (document or segment slot, head) pairs
};
// dirs: directions walked, each by dv / 64 workgroups in the backward.  Several documents take half
// shares there unless none of them is longer than a share: 4 ragged documents of 32768 tokens x 32
// heads 1576 -> 1296 us, but equal ones 1020 -> 1234 if cut like that.  The limit has no slack: four
// equal documents x 32 heads are just a share long, and one token more in one of them cuts all (8193,
// 8191, 8192, 8192 tokens: 1234; three documents are always cut, 1284).  The forward has its longest
// segments first instead (37 ragged documents, 16411 tokens, 32 heads with half shares 223 us, whole
// ones 208).
Plan walk_plan(const kda_linear_config* c, int64_t T, int32_t N, int dirs) {
    Plan p = {0, 0, (int64_t)N * c->H};
    const int64_t share = T * c->H * (dirs == 2 ? 2 * (c->dv / 64) : 1) / kWalkTarget;
    const double least = std::max(0.8 * dirs * sqrt((double)T * c->H * c->dk * c->dv) / 128.0, 1.4 * sqrt((double)T));
    int64_t floor = kLinBlock;
    while (floor < least) floor *= 2;
    auto length = [floor](int64_t share) { return std::max(floor, (share + kLinBlock - 1) / kLinBlock * kLinBlock); };
    const int64_t whole = length(share);
    if (T <= 2 * whole || T <= kWholeTokens || N > kSegDocs) return p;
    p.seg_len = (int32_t)(dirs == 2 && N > 1 ? length(share / 2) : whole);
    p.whole_len = p.seg_len == whole ? 0 : (int32_t)whole;
    p.chains = linear_slots(T, N, p.seg_len) * c->H;
    return p;
}

size_t elem(const kda_linear_config* c) { return c->in_dtype == KDA_BF16 ? 2 : 4; }
size_t state_elems(const kda_linear_config* c) { return (size_t)c->dk * c->dv; }

struct FwdLayout {
    Plan plan;
    size_t state, decay, total;
};
FwdLayout fwd_layout(const kda_linear_config* c, int64_t T, int32_t N) {
    FwdLayout f = {walk_plan(c, T, N, 1), 0, 0, 0};
    if (f.plan.seg_len) {
        f.decay = align256((size_t)f.plan.chains * state_elems(c) * sizeof(float));
        f.total = f.decay + align256((size_t)f.plan.chains * sizeof(float));
    }
    return f;
}

struct BwdLayout {
    Plan plan;
    int64_t blocks;
    int32_t parts;
    size_t S, dS, e, a, f, cross, part, sums, seg[2], decay[2], total;
};
// A key head's value heads are divided among so many workgroups: the smallest divisor of their
// number that gives kGradTarget workgroups (three roles a block), or the largest that does not,
// so that short streams do not wait for one workgroup's value heads in turn.  Backward in us, whole and divided for 256, 512
// and 1024 workgroups: 134 tokens x 8 heads on 2: 44, 27, 27, 27; 1024 x 32 on 8: 87, 87, 77,
// 81; 4096 x 16 on 4: 130, 130, 139, 143; 4096 x 32 on 1: 354, 192, 189, 186.  A prime number of
// value heads is divided into single ones, whole and so: 1152 x 28 on 4: 116, 97; 2048 x 28 on 4:
// 134, 131; 1024 x 127 on 1: 1144, 205.  (Workspace: two rows of dk fp32 a token and part.)
constexpr int64_t kGradTarget = 384;   // 288 workgroups gain from it (1024 x 32 on 8), 408 lose (4096 x 16 on 4)
int32_t grad_parts(const kda_linear_config* c, int64_t blocks) {
    const int32_t R = c->H / c->Hk;
    const int64_t groups = 3 * blocks * c->Hk;
    int32_t parts = 1;
    for (int32_t x = 2; x <= R && groups * parts < kGradTarget && x <= kGradTarget; ++x)
        if (R % x == 0) parts = x;
    return parts;
}
BwdLayout bwd_layout(const kda_linear_config* c, int64_t T, int32_t N) {
    BwdLayout b;
    memset(&b, 0, sizeof b);
    b.plan = walk_plan(c, T, N, 2);
    b.blocks = linear_slots(T, N, kLinBlock);
    b.parts = grad_parts(c, b.blocks);
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t x = at;
        at += align256(bytes);
        return x;
    };
    const size_t states = (size_t)b.blocks * c->H * state_elems(c) * elem(c), rows = (size_t)T * c->H * sizeof(float);
    b.S = take(states);
    b.dS = take(states);
    b.e = take(rows);
    b.a = take(rows);
    b.f = take(rows);
    b.cross = take((size_t)b.blocks * c->H * sizeof(float));
    b.part = take(gate_of(c) == KDA_GATE_HEAD ? (size_t)b.blocks * c->H * sizeof(float) : 0);
    b.sums = take(b.parts > 1 ? (size_t)2 * b.parts * T * c->Hk * c->dk * sizeof(float) : 0);
    if (b.plan.seg_len)
        for (int i = 0; i < 2; ++i) {
            b.seg[i] = take((size_t)b.plan.chains * state_elems(c) * sizeof(float));
            b.decay[i] = take((size_t)b.plan.chains * sizeof(float));
        }
    b.total = at;
    return b;
}

kda_status check_sizes(const kda_linear_config* c, int64_t T, int32_t N) {
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(KDA_ERR_INVALID_ARG, "total_tokens must be in [0, 2^31)%s");
    if (N < 1) return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 1%s");
    // the kernels address a block's rows with 32-bit byte offsets from a 64-bit base
    if ((int64_t)kLinBlock * c->H * 128 * 4 >= ((int64_t)1 << 31)) return fail(KDA_ERR_UNSUPPORTED, "H too large%s");
    // the largest launches: the walks' chains in at most four ways of kThreads, a block's gradients in at most three roles
    // a head, and the carry's at most four workgroups of kThreads for each of N * H states
    if (!grid_fits((linear_slots(T, N, kLinBlock) + 8) * 4 * (int64_t)c->H, kGradThreads))
        return fail(KDA_ERR_UNSUPPORTED, "num_seqs, H or total_tokens too large for one launch%s");
    return KDA_OK;
}
kda_status check_stream(const kda_linear_config* c, int64_t T, int32_t N, const int32_t* cu) {
    KDA_TRY(check_config(c));
    KDA_TRY(check_sizes(c, T, N));
    if (!cu && T % N) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens is NULL but total_tokens is not a multiple of num_seqs%s");
    return ptr(cu, "cu_seqlens", false);
}

bool overlap(const void* a, const void* b, size_t bytes) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + bytes && y < x + bytes;
}
// A step reads and writes each part of the state in one workgroup, so it may run in place.
kda_status check_step(const float* in, const float* out, size_t bytes) {
    if (in != out && overlap(in, out, bytes)) return fail(KDA_ERR_INVALID_ARG, "state_in and state_out overlap without being equal%s");
    return KDA_OK;
}

kda_status check_tree(const kda_tree_config* c, int32_t N, int threads, int64_t per_head) {
    if (!c) return fail(KDA_ERR_INVALID_ARG, "config is NULL%s");
    if (c->rule != KDA_RULE_DELTA && c->rule != KDA_RULE_LINEAR) return fail(KDA_ERR_INVALID_ARG, "unknown rule%s");
    KDA_TRY(check_heads(c->H, c->Hk, c->dk, c->dv, c->in_dtype, c->out_dtype, c->gate, c->scale));
    if (c->rule == KDA_RULE_DELTA && (c->Hk != c->H || c->gate != KDA_GATE_TOKEN))
        return fail(KDA_ERR_UNSUPPORTED, "the delta rule has Hk = H and a gate per token%s");
    if (!(c->l2_eps >= 0.f) || !isfinite(c->l2_eps)) return fail(KDA_ERR_INVALID_ARG, "l2_eps must be finite and >= 0%s");
    if (c->nodes < 1 || c->nodes > KDA_TREE_MAX_NODES) return fail(KDA_ERR_UNSUPPORTED, "nodes must be in [1, 64]%s");
    if (N < 0) return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 0%s");
    if (!grid_fits((int64_t)N * c->H * per_head, threads)) return fail(KDA_ERR_UNSUPPORTED, "num_seqs * H too large for one launch%s");
    return KDA_OK;
}
TreeParams tree_params(const kda_tree_config* c, int32_t N) {
    TreeParams p;
    memset(&p, 0, sizeof p);
    p.N = N; p.H = c->H; p.Hk = c->Hk; p.L = c->nodes; p.dv = c->dv;
    p.gate_head = c->gate == KDA_GATE_HEAD;
    p.out_bf16 = c->out_dtype == KDA_BF16;
    p.eps = c->l2_eps; p.scale = c->scale;
    return p;
}

}  // namespace

static_assert(KDA_TREE_MAX_NODES == kda::kTreeMaxNodes, "tree size");

extern "C" {

void kda_linear_config_init(kda_linear_config* cfg, int32_t H, int32_t Hk, int32_t dk, int32_t dv) {
    if (!cfg) return;
    memset(cfg, 0, sizeof *cfg);
    cfg->H = H; cfg->Hk = Hk; cfg->dk = dk; cfg->dv = dv;
    cfg->in_dtype = KDA_F32; cfg->out_dtype = KDA_F32;
    cfg->gate = KDA_GATE_TOKEN;
    cfg->scale = 1.0f;
}

size_t kda_linear_fwd_workspace_size(const kda_linear_config* cfg, int64_t T, int32_t N) {
    if (check_config(cfg) != KDA_OK || check_sizes(cfg, T, N) != KDA_OK) return 0;
    return fwd_layout(cfg, T, N).total;
}

size_t kda_linear_bwd_workspace_size(const kda_linear_config* cfg, int64_t T, int32_t N) {
    if (check_config(cfg) != KDA_OK || check_sizes(cfg, T, N) != KDA_OK) return 0;
    return bwd_layout(cfg, T, N).total;
}

kda_status kda_linear_fwd(const kda_linear_config* cfg, int64_t T, int32_t N, const void* q, const void* k, const void* v,
                          const float* g, const int32_t* cu, const float* s0, void* o, float* sfinal, void* workspace,
                          size_t workspace_bytes, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_stream(cfg, T, N, cu));
    KDA_TRY(ptr(q, "q", T > 0));
    KDA_TRY(ptr(k, "k", T > 0));
    KDA_TRY(ptr(v, "v", T > 0));
    KDA_TRY(ptr(g, "g", T > 0));
    KDA_TRY(ptr(o, "o", T > 0));
    KDA_TRY(ptr(s0, "initial_state", false));
    KDA_TRY(ptr(sfinal, "final_state", false));
    // A document's last segment may write its state before the first has read its own.
    if (overlap(s0, sfinal, (size_t)N * cfg->H * state_elems(cfg) * sizeof(float)))
        return fail(KDA_ERR_INVALID_ARG, "final_state overlaps initial_state%s");
    const FwdLayout f = fwd_layout(cfg, T, N);
    if (workspace_bytes < f.total) return fail(KDA_ERR_WORKSPACE, "workspace too small%s");
    KDA_TRY(ptr(workspace, "workspace", f.total > 0));

    hipStream_t st = (hipStream_t)stream;
    LinearParams p;
    memset(&p, 0, sizeof p);
    p.q = q; p.k = k; p.v = v; p.g = g; p.cu = cu; p.s0 = s0; p.o = o; p.sfinal = sfinal;
    p.T = T; p.N = N; p.H = cfg->H; p.Hk = cfg->Hk; p.dv = cfg->dv;
    p.seqlen = cu ? 0 : (int32_t)(T / N);
    p.g_stride = gate_of(cfg) == KDA_GATE_TOKEN ? cfg->H : 0;
    p.out_bf16 = cfg->out_dtype == KDA_BF16;
    p.scale = cfg->scale;
    p.seg_len = f.plan.seg_len;
    p.chains = (int32_t)f.plan.chains;
    if (p.seg_len) {
        float* state = (float*)workspace;
        float* decay = (float*)((char*)workspace + f.decay);
        LinearStateParams s;
        memset(&s, 0, sizeof s);
        s.dir[0].a = k; s.dir[0].b = v; s.dir[0].seg = state; s.dir[0].decay = decay;
        s.g = g; s.cu = cu; s.T = T; s.N = N; s.H = p.H; s.Hk = p.Hk; s.dv = p.dv; s.seqlen = p.seqlen;
        s.g_stride = p.g_stride; s.seg_len = p.seg_len; s.chains = p.chains; s.dirs = 1; s.scale = p.scale;
        KDA_TRY(launched(launch_linear_states(s, cfg->in_dtype, cfg->dk, st)));
        LinearCarryParams c;
        memset(&c, 0, sizeof c);
        c.dir[0].s0 = s0; c.dir[0].seg = state; c.dir[0].decay = decay;
        c.cu = cu; c.T = T; c.N = N; c.H = p.H; c.seqlen = p.seqlen; c.seg_len = p.seg_len; c.elems = cfg->dk * cfg->dv; c.slots = (int32_t)linear_slots(T, N, p.seg_len);
        KDA_TRY(launched(launch_linear_carry(c, 1, st)));
        p.seg_state = state;
        // Longest first where workgroups follow one another (37 ragged documents, 16411 tokens, 32
        // heads: 236 -> 226 us; 64, 16384, 16: 158 -> 142).  Where all run at once it only costs (25,
        // 6229, 4: 36 -> 40).  A wave looks for the order among its lanes, so at most 64 documents.
        p.longest_first = N > 1 && N <= 64 && f.plan.chains > kWalkTarget;
    }
    return launched(launch_linear_out(p, cfg->in_dtype, cfg->dk, st));
}

kda_status kda_linear_bwd(const kda_linear_config* cfg, int64_t T, int32_t N, const void* q, const void* k, const void* v,
                          const float* g, const int32_t* cu, const float* s0, const void* dO, const float* dSf, void* dq,
                          void* dk, void* dv, void* dg, float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_stream(cfg, T, N, cu));
    const bool any = T > 0;
    KDA_TRY(ptr(q, "q", any));
    KDA_TRY(ptr(k, "k", any));
    KDA_TRY(ptr(v, "v", any));
    KDA_TRY(ptr(g, "g", any));
    KDA_TRY(ptr(dO, "dO", any));
    KDA_TRY(ptr(dq, "dq", any));
    KDA_TRY(ptr(dk, "dk", any));
    KDA_TRY(ptr(dv, "dv", any));
    KDA_TRY(ptr(dg, "dg", any || gate_of(cfg) == KDA_GATE_HEAD));
    KDA_TRY(ptr(s0, "initial_state", false));
    KDA_TRY(ptr(dSf, "dS_final", false));
    KDA_TRY(ptr(dS0, "d_initial_state", false));
    // One launch walks both ways: the reverse walk's end writes what either walk's start may still have to read.
    const size_t states = (size_t)N * cfg->H * state_elems(cfg) * sizeof(float);
    if (overlap(dS0, s0, states)) return fail(KDA_ERR_INVALID_ARG, "d_initial_state overlaps initial_state%s");
    if (overlap(dS0, dSf, states)) return fail(KDA_ERR_INVALID_ARG, "d_initial_state overlaps dS_final%s");
    const BwdLayout b = bwd_layout(cfg, T, N);
    if (workspace_bytes < b.total) return fail(KDA_ERR_WORKSPACE, "workspace too small%s");
    KDA_TRY(ptr(workspace, "workspace", b.total > 0));

    hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    const int32_t seqlen = cu ? 0 : (int32_t)(T / N), g_stride = gate_of(cfg) == KDA_GATE_TOKEN ? cfg->H : 0;
    LinearStateParams s;
    memset(&s, 0, sizeof s);
    s.dir[0].a = k; s.dir[0].b = v;
    s.dir[1].a = q; s.dir[1].b = dO; s.dir[1].rev = 1;
    s.g = g; s.cu = cu; s.T = T; s.N = N; s.H = cfg->H; s.Hk = cfg->Hk; s.dv = cfg->dv; s.seqlen = seqlen;
    s.g_stride = g_stride; s.seg_len = b.plan.seg_len; s.whole_len = b.plan.whole_len; s.chains = (int32_t)b.plan.chains; s.dirs = 2; s.scale = cfg->scale;
    const float* first[2] = {s0, dSf};
    float* last[2] = {nullptr, dS0};
    if (s.seg_len) {
        LinearCarryParams c;
        memset(&c, 0, sizeof c);
        for (int i = 0; i < 2; ++i) {
            s.dir[i].seg = (float*)(ws + b.seg[i]);
            s.dir[i].decay = (float*)(ws + b.decay[i]);
            c.dir[i].s0 = first[i]; c.dir[i].seg = s.dir[i].seg; c.dir[i].decay = s.dir[i].decay; c.dir[i].rev = i;
        }
        c.cu = cu; c.T = T; c.N = N; c.H = cfg->H; c.seqlen = seqlen; c.seg_len = s.seg_len; c.whole_len = s.whole_len; c.elems = cfg->dk * cfg->dv;
        c.slots = (int32_t)linear_slots(T, N, s.seg_len);
        KDA_TRY(launched(launch_linear_states(s, cfg->in_dtype, cfg->dk, st)));
        KDA_TRY(launched(launch_linear_carry(c, 2, st)));
    }
    for (int i = 0; i < 2; ++i) {
        s.dir[i].s0 = first[i];
        s.dir[i].last = last[i];
        s.dir[i].decay = nullptr;
    }
    s.dir[0].border = ws + b.S;
    s.dir[1].border = ws + b.dS;
    KDA_TRY(launched(launch_linear_states(s, cfg->in_dtype, cfg->dk, st)));

    LinearBwdParams p;
    memset(&p, 0, sizeof p);
    p.q = q; p.k = k; p.v = v; p.g = g; p.cu = cu; p.dO = dO;
    p.S = ws + b.S; p.dS = ws + b.dS;
    p.e = (float*)(ws + b.e); p.a = (float*)(ws + b.a); p.f = (float*)(ws + b.f); p.cross = (float*)(ws + b.cross);
    p.dg_part = gate_of(cfg) == KDA_GATE_HEAD ? (float*)(ws + b.part) : nullptr;
    p.sums = (float*)(ws + b.sums); p.parts = b.parts;
    p.dq = dq; p.dk_out = dk; p.dv_out = dv; p.dg = dg;
    p.T = T; p.blocks = T > 0 ? b.blocks : 0; p.N = N; p.H = cfg->H; p.Hk = cfg->Hk; p.dv = cfg->dv; p.seqlen = seqlen;
    p.g_stride = g_stride; p.out_bf16 = cfg->out_dtype == KDA_BF16;
    p.dg_bf16 = p.out_bf16 && !(cfg->gate & KDA_GATE_GRAD_F32);
    p.scale = cfg->scale;
    return launched(launch_linear_grads(p, cfg->in_dtype, cfg->dk, st));
}

kda_status kda_linear_decode(const kda_linear_config* cfg, int32_t N, const void* q, const void* k, const void* v,
                             const float* g, const float* state_in, float* state_out, void* o, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_config(cfg));
    if (N < 0) return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 0%s");
    if (!grid_fits((int64_t)N * cfg->H * (cfg->dv / kSlice), kThreads))
        return fail(KDA_ERR_UNSUPPORTED, "num_seqs * H too large for one launch%s");
    KDA_TRY(ptr(q, "q", N > 0));
    KDA_TRY(ptr(k, "k", N > 0));
    KDA_TRY(ptr(v, "v", N > 0));
    KDA_TRY(ptr(g, "g", N > 0));
    KDA_TRY(ptr(state_in, "state_in", false));
    KDA_TRY(ptr(state_out, "state_out", N > 0));
    KDA_TRY(ptr(o, "o", N > 0));
    KDA_TRY(check_step(state_in, state_out, (size_t)N * cfg->H * state_elems(cfg) * sizeof(float)));
    LinearDecodeParams p;
    memset(&p, 0, sizeof p);
    p.q = q; p.k = k; p.v = v; p.g = g; p.s_in = state_in; p.s_out = state_out; p.o = o;
    p.N = N; p.H = cfg->H; p.Hk = cfg->Hk; p.dv = cfg->dv;
    p.g_stride = gate_of(cfg) == KDA_GATE_TOKEN ? cfg->H : 0;
    p.out_bf16 = cfg->out_dtype == KDA_BF16;
    p.scale = cfg->scale;
    return launched(launch_linear_decode(p, cfg->in_dtype, cfg->dk, (hipStream_t)stream));
}

void kda_tree_config_init(kda_tree_config* cfg, int32_t rule, int32_t H, int32_t Hk, int32_t dk, int32_t dv, int32_t nodes) {
    if (!cfg) return;
    memset(cfg, 0, sizeof *cfg);
    cfg->rule = rule; cfg->H = H; cfg->Hk = Hk; cfg->dk = dk; cfg->dv = dv; cfg->nodes = nodes;
    cfg->in_dtype = KDA_F32; cfg->out_dtype = KDA_F32;
    cfg->gate = KDA_GATE_TOKEN;
    cfg->l2_eps = 1e-6f;
    cfg->scale = 1.0f;
}

kda_status kda_tree(const kda_tree_config* cfg, int32_t N, const void* q, const void* k, const void* v, const void* g,
                    const void* beta, const int32_t* parent, const float* state, void* o, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_tree(cfg, N, 512, 1));
    const bool delta = cfg->rule == KDA_RULE_DELTA;
    KDA_TRY(ptr(q, "q", N > 0));
    KDA_TRY(ptr(k, "k", N > 0));
    KDA_TRY(ptr(v, "v", N > 0));
    KDA_TRY(ptr(g, "g", N > 0));
    KDA_TRY(ptr(beta, "beta", N > 0 && delta));
    KDA_TRY(ptr(parent, "parent", N > 0));
    KDA_TRY(ptr(state, "state", false));
    KDA_TRY(ptr(o, "o", N > 0));
    TreeParams p = tree_params(cfg, N);
    p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.parent = parent; p.s_in = state; p.o = o;
    return launched(launch_tree(p, delta, cfg->in_dtype, cfg->dk, (hipStream_t)stream));
}

kda_status kda_tree_commit(const kda_tree_config* cfg, int32_t N, const void* k, const void* v, const void* g,
                           const void* beta, const int32_t* parent, const int32_t* accept, const float* state_in,
                           float* state_out, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_tree(cfg, N, kThreads, cfg ? cfg->dv / kSlice : 1));
    const bool delta = cfg->rule == KDA_RULE_DELTA;
    KDA_TRY(ptr(k, "k", N > 0));
    KDA_TRY(ptr(v, "v", N > 0));
    KDA_TRY(ptr(g, "g", N > 0));
    KDA_TRY(ptr(beta, "beta", N > 0 && delta));
    KDA_TRY(ptr(parent, "parent", N > 0));
    KDA_TRY(ptr(accept, "accept", N > 0));
    KDA_TRY(ptr(state_in, "state_in", false));
    KDA_TRY(ptr(state_out, "state_out", N > 0));
    KDA_TRY(check_step(state_in, state_out, (size_t)N * cfg->H * cfg->dk * cfg->dv * sizeof(float)));
    TreeParams p = tree_params(cfg, N);
    p.k = k; p.v = v; p.g = g; p.beta = beta; p.parent = parent; p.accept = accept;
    p.s_in = state_in; p.s_out = state_out;
    return launched(launch_tree_commit(p, delta, cfg->in_dtype, cfg->dk, (hipStream_t)stream));
}

}  // extern "C"
