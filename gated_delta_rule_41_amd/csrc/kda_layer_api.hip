// kda_layer_api.hip -- the C ABI of the norm, the short convolution and the selective scan
// (include/kda.h).  As in kda_api.hip every argument is checked on the host before any HIP
// call, and nothing is allocated.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/kda.h"
#include "kda_internal.h"
#include "kda_layer.h"

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
size_t elem(int32_t t) { return t == KDA_F32 ? 4 : t == KDA_BF16 ? 2 : 1; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}
kda_status apart(const void* a, size_t na, const char* name, const void* b, size_t nb) {
    return overlap(a, na, b, nb) ? fail(KDA_ERR_INVALID_ARG, "%s overlaps another argument", name) : KDA_OK;
}
// An argument's memory.  An output may lie in memory of its own only, or be an input of its `kind` itself, of the same bytes.
struct Span {
    const void* p;
    size_t bytes;
    const char* name;
    int kind;                                     // 0: shared with nothing
};
constexpr int kRowsOf = 1, kStates = 2, kMostSpans = 24;
kda_status outputs_apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    // all pairs without a branch first: a small call's launch takes microseconds, this some tenths of one
    uintptr_t from[kMostSpans], to[kMostSpans];
    int n = 0;
    for (const auto* list : {&inputs, &outputs})
        for (const Span& x : *list) {
            from[n] = (uintptr_t)x.p;
            to[n++] = x.p ? (uintptr_t)x.p + x.bytes : 0;
        }
    unsigned any = 0;
    for (int o = (int)inputs.size(); o < n; ++o)
        for (int i = 0; i < o; ++i) any |= (unsigned)(from[o] < to[i]) & (unsigned)(from[i] < to[o]);
    if (!any) return KDA_OK;
    for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span& i : inputs)
            if (!(o->kind && o->kind == i.kind && o->p == i.p && o->bytes == i.bytes)) KDA_TRY(apart(o->p, o->bytes, o->name, i.p, i.bytes));
        for (const Span* other = outputs.begin(); other != o; ++other) KDA_TRY(apart(o->p, o->bytes, o->name, other->p, other->bytes));
    }
    return KDA_OK;
}
// The largest number of workgroups along x: one launch covers at most 2^32 - 1 work-items.
bool grid_fits(int64_t workgroups, int threads) { return workgroups >= 0 && workgroups <= (int64_t)UINT32_MAX / threads; }

kda_status check_sizes(int64_t T, int32_t N) {
    if (T < 0 || T >= ((int64_t)1 << 31)) return fail(KDA_ERR_INVALID_ARG, "total_tokens must be in [0, 2^31)%s");
    if (N < 1) return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 1%s");
    return KDA_OK;
}
kda_status check_stream(int64_t T, int32_t N, const int32_t* cu) {
    if (!cu && T % N) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens is NULL but total_tokens is not a multiple of num_seqs%s");
    return ptr(cu, "cu_seqlens", false);
}

// ---------------------------------------------------------------- norm
kda_status check_norm(const kda_norm_config* c, int64_t rows, bool backward) {
    if (!c) return fail(KDA_ERR_INVALID_ARG, "config is NULL%s");
    if (c->C < 1) return fail(KDA_ERR_INVALID_ARG, "C must be >= 1%s");
    if (c->C > KDA_NORM_MAX_CHANNELS) return fail(KDA_ERR_UNSUPPORTED, "C too large%s");
    if (!is_dtype(c->in_dtype) || !is_dtype(c->res_dtype) || !is_dtype(c->weight_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype%s");
    if (!is_dtype(c->out_dtype) && (backward || (c->out_dtype != KDA_I8 && c->out_dtype != KDA_E4M3)))
        return fail(KDA_ERR_INVALID_ARG, "unknown output dtype%s");
    if (c->in_dtype == KDA_F32 && c->res_dtype == KDA_BF16) return fail(KDA_ERR_UNSUPPORTED, "fp32 inputs take an fp32 residual%s");
    if (!(c->eps >= 0.f) || !isfinite(c->eps)) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0%s");
    if (rows < 0) return fail(KDA_ERR_INVALID_ARG, "rows must be >= 0%s");
    // the forward's launch; the backward's workgroups take as many rows as there are
    const int at_once = norm_fwd_rows(c->C);
    if (!grid_fits(rows / at_once + (rows % at_once != 0), norm_fwd_threads(c->C)))
        return fail(KDA_ERR_UNSUPPORTED, "rows too large for one launch%s");
    return KDA_OK;
}

// ---------------------------------------------------------------- convolution
kda_status check_conv(const kda_conv_config* c) {
    if (!c) return fail(KDA_ERR_INVALID_ARG, "config is NULL%s");
    if (c->C < 1) return fail(KDA_ERR_INVALID_ARG, "C must be >= 1%s");
    if (c->C > KDA_CONV_MAX_CHANNELS) return fail(KDA_ERR_UNSUPPORTED, "C too large%s");
    if (c->width < 2 || c->width > 4) return fail(KDA_ERR_UNSUPPORTED, "width must be 2, 3 or 4%s");
    if (!is_dtype(c->in_dtype) || !is_dtype(c->out_dtype) || !is_dtype(c->weight_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype%s");
    if (c->activation != KDA_ACT_NONE && c->activation != KDA_ACT_SILU) return fail(KDA_ERR_INVALID_ARG, "unknown activation%s");
    if (c->x_stride != 0 && c->x_stride < c->C) return fail(KDA_ERR_INVALID_ARG, "x_stride is below C%s");
    return KDA_OK;
}
int64_t row_stride(int64_t stride, int64_t width) { return stride ? stride : width; }
size_t cu_bytes(int32_t N) { return ((size_t)N + 1) * sizeof(int32_t); }
// From the first element to the last, in bytes.
size_t extent(int64_t rows, int64_t stride, int64_t width, size_t es) { return rows > 0 ? ((size_t)(rows - 1) * stride + width) * es : 0; }

// Channels a thread: eight move whole 16-byte pieces, one gives small calls eight times the threads, each with an eighth
// to do.  One rule for both directions, by the sum of the two.  us of a forward and a backward, eight and one, width 4:
// bf16 1000 x 512 5.0, 16.0 and 4.0, 10.6;  1000 x 2048 5.4, 18.6 and 5.7, 13.3;  16000 x 333 7.8, 29.2 and 8.6, 27.1;
// 1000 x 8192 7.3, 27.1 and 9.5, 32.3;  fp32 4000 x 2048 16.9, 36.5 and 15.5, 32.9;  16000 x 2048 54.1, 93.5 and 45.6,
// 106.8: there a forward by itself would gain from one.
bool conv_eight(const kda_conv_config* c, int64_t T) {
    return c->C >= 8 && T * c->C >= (c->in_dtype == KDA_BF16 ? (int64_t)1 << 22 : (int64_t)1 << 24);
}
// Tokens a strip.  A strip begins with W - 1 rows and the taps, and in the backward ends with its sums; many strips
// even out.  us for 8, 16, 32, 64, 96, 128, 192 tokens: forward of 16411 x 12288 168, 157, 167, 179, 191, 199, 203;
// backward of 32768 x 4096 362, 263, 225, 182, 232, 166, 218, where 64 and 128 are two and one wave a SIMD's two
// registers' worth, so strips there make whole rounds of 2048 waves.
int32_t conv_len(const kda_conv_config* c, int64_t T, bool backward) {
    const int64_t per = conv_eight(c, T) ? (c->C + 7) / 8 : c->C;
    const int64_t share = T * per / (64 * 2048);      // tokens a wave in one round
    if (share < 16) return share < 8 ? 8 : 16;
    if (!backward) return 16;
    const int64_t rounds = (share + 127) / 128;
    return (int32_t)((share + rounds - 1) / rounds);
}
kda_status conv_plan(const kda_conv_config* c, int64_t T, int32_t N, bool backward, int32_t* len, int64_t* slots) {
    *len = conv_len(c, T, backward);
    *slots = layer_slots(T, N, *len);
    return grid_fits(*slots, kLayerThreads) ? KDA_OK : fail(KDA_ERR_UNSUPPORTED, "num_seqs or total_tokens too large for one launch%s");
}
size_t conv_state(const kda_conv_config* c, int32_t N) { return (size_t)N * (c->width - 1) * c->C * elem(c->in_dtype); }
size_t conv_weights(const kda_conv_config* c) { return (size_t)c->C * c->width * elem(c->weight_dtype); }
size_t conv_bias(const kda_conv_config* c) { return c->C * elem(c->weight_dtype); }
ConvParams conv_params(const kda_conv_config* c) {
    ConvParams p;
    memset(&p, 0, sizeof p);
    p.C = c->C;
    p.x_stride = row_stride(c->x_stride, c->C);
    p.out_bf16 = c->out_dtype == KDA_BF16;
    p.weight_bf16 = c->weight_dtype == KDA_BF16;
    p.silu = c->activation == KDA_ACT_SILU;
    return p;
}

// ---------------------------------------------------------------- selective scan
kda_status check_selective(const kda_selective_config* c) {
    if (!c) return fail(KDA_ERR_INVALID_ARG, "config is NULL%s");
    if (c->C < 1 || c->G < 1 || c->C % c->G) return fail(KDA_ERR_INVALID_ARG, "C and G must be >= 1 and G must divide C%s");
    if (c->C > KDA_SELECTIVE_MAX_CHANNELS) return fail(KDA_ERR_UNSUPPORTED, "C too large%s");
    if (c->S != 8 && c->S != 16 && c->S != 32) return fail(KDA_ERR_UNSUPPORTED, "S must be 8, 16 or 32%s");
    if (!is_dtype(c->in_dtype) || !is_dtype(c->out_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype%s");
    if (c->flags & ~KDA_SELECTIVE_SOFTPLUS) return fail(KDA_ERR_INVALID_ARG, "unknown flags%s");
    const int64_t strides[3] = {c->x_stride, c->dt_stride, c->z_stride};
    for (int64_t s : strides)
        if (s != 0 && s < c->C) return fail(KDA_ERR_INVALID_ARG, "a row stride is below C%s");
    const int64_t rows[2] = {c->b_stride, c->c_stride};
    for (int64_t s : rows) {
        if (s != 0 && s < (int64_t)c->G * c->S) return fail(KDA_ERR_INVALID_ARG, "a row stride of B or C is below G * S%s");
        if (s * elem(c->in_dtype) % 16) return fail(KDA_ERR_UNSUPPORTED, "row strides of B and C must be multiples of 16 bytes%s");
    }
    return KDA_OK;
}
int32_t group_waves(const kda_selective_config* c) { return (c->C / c->G + 63) / 64; }

// Segments are short: their waves even out over the compute units, and a document's latency is a segment's
// walk and the steps of its carry.  Tokens a segment and us (37 ragged documents, 16411 tokens x 4096 channels;
// 131083 x 512; backward of 4 x 4096 x 4096):  48: 488, 490, 1429;  96: 467, 458, 1389;  144: 500, 494, 1484;
// 528: 822, 605, 2572.  kSelectiveWaves makes that about 96.  Short streams: a backward of 1003 tokens x 200
// channels takes 64 us at 12, 82 at 24 and 129 at 48; the root is where a token's walk (0.8 us alone) and its
// share of the carry (0.05 us a segment) are equal.
constexpr int64_t kSelectiveWaves = 10922;
constexpr int64_t kSelectiveUnit = 12;      // tokens; whole kept blocks at 8 and 16 entries
struct SelectivePlan {
    int64_t len, slots, borders;
    bool cut;
    size_t seg, sdt, rseg, border, bdt, bc, par, total;
};
// cu_seqlens is on the device, so any document may have all the tokens.
SelectivePlan selective_plan(const kda_selective_config* c, int64_t T, int32_t N, bool backward) {
    SelectivePlan p;
    memset(&p, 0, sizeof p);
    auto up = [](int64_t x) { return std::max(kSelectiveUnit, (x + kSelectiveUnit - 1) / kSelectiveUnit * kSelectiveUnit); };
    const int64_t waves = (int64_t)group_waves(c) * c->G;
    p.len = up(std::max(T * waves / kSelectiveWaves, (int64_t)sqrt((double)T / 16)));
    p.cut = T > p.len;
    if (!p.cut) p.len = up(T);
    p.slots = layer_slots(T, N, (int32_t)p.len);
    const size_t states = (size_t)p.slots * c->C * c->S * sizeof(float), sums = (size_t)p.slots * c->C * sizeof(float);
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t x = at;
        at += align256(bytes);
        return x;
    };
    if (p.cut || backward) {
        p.seg = take(states);
        p.sdt = take(sums);
    }
    if (backward) {
        p.borders = T / selective_kept(c->S) + N;
        p.rseg = take(p.cut ? states : 0);
        p.border = take((size_t)p.borders * c->C * c->S * sizeof(float));
        p.bdt = take((size_t)p.borders * c->C * sizeof(float));
        p.bc = take((size_t)T * waves * 2 * c->S * sizeof(float));
        p.par = take((size_t)p.slots * c->C * (c->S + 2) * sizeof(float));
    }
    p.total = at;
    return p;
}
kda_status check_selective_sizes(const kda_selective_config* c, int64_t T, int32_t N) {
    KDA_TRY(check_sizes(T, N));
    const SelectivePlan p = selective_plan(c, T, N, false);
    if (!grid_fits(p.slots, kLayerThreads) || !grid_fits((T * c->G * 2 * c->S + kLayerThreads - 1) / kLayerThreads, kLayerThreads))
        return fail(KDA_ERR_UNSUPPORTED, "num_seqs or total_tokens too large for one launch%s");
    return KDA_OK;
}
// Bytes of the arguments, T rows of each.
struct SelectiveSizes {
    size_t x, dt, z, dy, out, B, C, dB, A, D, state;
    int in_place;                                 // outputs of rows may be inputs of rows
    SelectiveSizes(const kda_selective_config* c, int64_t T, int32_t N) {
        const size_t es = elem(c->in_dtype), os = elem(c->out_dtype);
        const int64_t gs = (int64_t)c->G * c->S;
        x = extent(T, row_stride(c->x_stride, c->C), c->C, es);
        dt = extent(T, row_stride(c->dt_stride, c->C), c->C, es);
        z = extent(T, row_stride(c->z_stride, c->C), c->C, es);
        dy = extent(T, c->C, c->C, es);
        out = extent(T, c->C, c->C, os);
        B = extent(T, row_stride(c->b_stride, gs), gs, es);
        C = extent(T, row_stride(c->c_stride, gs), gs, es);
        dB = extent(T, gs, gs, os);
        A = (size_t)c->C * c->S * sizeof(float);
        D = c->C * sizeof(float);
        state = N * A;
        in_place = es == os ? kRowsOf : 0;
    }
};
SelectiveParams selective_params(const kda_selective_config* c) {
    SelectiveParams p;
    memset(&p, 0, sizeof p);
    p.C = c->C; p.G = c->G;
    p.x_stride = row_stride(c->x_stride, c->C);
    p.dt_stride = row_stride(c->dt_stride, c->C);
    p.z_stride = row_stride(c->z_stride, c->C);
    p.b_stride = row_stride(c->b_stride, (int64_t)c->G * c->S);
    p.c_stride = row_stride(c->c_stride, (int64_t)c->G * c->S);
    p.out_bf16 = c->out_dtype == KDA_BF16;
    p.softplus = (c->flags & KDA_SELECTIVE_SOFTPLUS) != 0;
    p.group_waves = group_waves(c);
    p.waves = p.group_waves * c->G;
    return p;
}

}  // namespace

extern "C" {

void kda_norm_config_init(kda_norm_config* cfg, int32_t C) {
    if (!cfg) return;
    memset(cfg, 0, sizeof *cfg);
    cfg->C = C;
    cfg->eps = 1e-6f;
}

kda_status kda_norm_fwd(const kda_norm_config* cfg, int64_t rows, const void* x, const void* residual, const void* weight,
                        void* y, void* s, float* scale, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_norm(cfg, rows, false));
    const bool any = rows > 0, codes = !is_dtype(cfg->out_dtype);
    if (!residual && cfg->res_dtype != cfg->in_dtype) return fail(KDA_ERR_INVALID_ARG, "res_dtype must be in_dtype without a residual%s");
    KDA_TRY(ptr(x, "x", any));
    KDA_TRY(ptr(residual, "residual", false));
    KDA_TRY(ptr(weight, "weight", false));
    KDA_TRY(ptr(y, "y", any));
    KDA_TRY(ptr(s, "s", false));
    KDA_TRY(ptr(scale, "scale", any && codes));
    if (!residual) s = nullptr;
    const size_t n = (size_t)rows * cfg->C, nx = n * elem(cfg->in_dtype), nr = n * elem(cfg->res_dtype), ny = n * elem(cfg->out_dtype);
    const size_t nw = cfg->C * elem(cfg->weight_dtype), ns = codes ? rows * sizeof(float) : 0;
    // every thread reads its part of a row before it writes it, so that equal pointers of one type are fine
    if (!(y == x && cfg->out_dtype == cfg->in_dtype)) KDA_TRY(apart(y, ny, "y", x, nx));
    KDA_TRY(apart(y, ny, "y", residual, nr));
    KDA_TRY(apart(y, ny, "y", s, nr));
    KDA_TRY(apart(y, ny, "y", weight, nw));
    if (!(s == x && cfg->res_dtype == cfg->in_dtype)) KDA_TRY(apart(s, nr, "s", x, nx));
    if (s != residual) KDA_TRY(apart(s, nr, "s", residual, nr));
    KDA_TRY(apart(s, nr, "s", weight, nw));
    if (codes) {
        KDA_TRY(apart(scale, ns, "scale", x, nx));
        KDA_TRY(apart(scale, ns, "scale", residual, nr));
        KDA_TRY(apart(scale, ns, "scale", weight, nw));
        KDA_TRY(apart(scale, ns, "scale", y, ny));
        KDA_TRY(apart(scale, ns, "scale", s, nr));
    }
    if (!any) return KDA_OK;
    NormParams p;
    memset(&p, 0, sizeof p);
    p.x = x; p.residual = residual; p.weight = weight; p.y = y; p.s = s; p.scale = scale;
    p.rows = rows; p.C = cfg->C; p.out = cfg->out_dtype; p.weight_bf16 = cfg->weight_dtype == KDA_BF16; p.eps = cfg->eps;
    return launched(launch_norm_fwd(p, cfg->in_dtype == KDA_BF16, cfg->res_dtype == KDA_BF16, (hipStream_t)stream));
}

size_t kda_norm_bwd_workspace_size(const kda_norm_config* cfg, int64_t rows) {
    if (check_norm(cfg, rows, true) != KDA_OK) return 0;
    return (size_t)norm_bwd_blocks(cfg->C, rows) * cfg->C * sizeof(float);
}

kda_status kda_norm_bwd(const kda_norm_config* cfg, int64_t rows, const void* s, const void* weight, const void* dy,
                        const void* ds, void* dx, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_norm(cfg, rows, true));
    const bool any = rows > 0;
    KDA_TRY(ptr(s, "s", any));
    KDA_TRY(ptr(weight, "weight", false));
    KDA_TRY(ptr(dy, "dy", any));
    KDA_TRY(ptr(ds, "ds", false));
    KDA_TRY(ptr(dx, "dx", any));
    KDA_TRY(ptr(dw, "dweight", false));
    const size_t n = (size_t)rows * cfg->C, nr = n * elem(cfg->res_dtype), ny = n * elem(cfg->in_dtype), nx = n * elem(cfg->out_dtype);
    const size_t nw = cfg->C * elem(cfg->weight_dtype), nd = cfg->C * sizeof(float);
    KDA_TRY(apart(dx, nx, "dx", s, nr));
    KDA_TRY(apart(dx, nx, "dx", weight, nw));
    if (!(dx == dy && cfg->out_dtype == cfg->in_dtype)) KDA_TRY(apart(dx, nx, "dx", dy, ny));
    if (!(dx == ds && cfg->out_dtype == cfg->res_dtype)) KDA_TRY(apart(dx, nx, "dx", ds, nr));
    KDA_TRY(apart(dw, nd, "dweight", s, nr));
    KDA_TRY(apart(dw, nd, "dweight", weight, nw));
    KDA_TRY(apart(dw, nd, "dweight", dy, ny));
    KDA_TRY(apart(dw, nd, "dweight", ds, nr));
    KDA_TRY(apart(dw, nd, "dweight", dx, nx));
    const size_t need = dw ? kda_norm_bwd_workspace_size(cfg, rows) : 0;
    if (workspace_bytes < need) return fail(KDA_ERR_WORKSPACE, "workspace too small%s");
    KDA_TRY(ptr(workspace, "workspace", need > 0));
    NormParams p;
    memset(&p, 0, sizeof p);
    p.x = s; p.weight = weight; p.dy = dy; p.ds = ds; p.dx = dx; p.dw_part = dw ? (float*)workspace : nullptr;
    p.rows = rows; p.C = cfg->C; p.out = cfg->out_dtype; p.weight_bf16 = cfg->weight_dtype == KDA_BF16; p.eps = cfg->eps;
    return launched(launch_norm_bwd(p, cfg->in_dtype == KDA_BF16, cfg->res_dtype == KDA_BF16, dw, (hipStream_t)stream));
}

void kda_conv_config_init(kda_conv_config* cfg, int32_t C, int32_t width) {
    if (!cfg) return;
    memset(cfg, 0, sizeof *cfg);
    cfg->C = C;
    cfg->width = width;
    cfg->activation = KDA_ACT_SILU;
}

kda_status kda_conv_fwd(const kda_conv_config* cfg, int64_t T, int32_t N, const void* x, const void* weight, const void* bias,
                        const int32_t* cu, const void* s0, void* y, void* sfinal, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_conv(cfg));
    KDA_TRY(check_sizes(T, N));
    KDA_TRY(check_stream(T, N, cu));
    KDA_TRY(ptr(x, "x", T > 0));
    KDA_TRY(ptr(weight, "weight", true));
    KDA_TRY(ptr(bias, "bias", false));
    KDA_TRY(ptr(s0, "initial_state", false));
    KDA_TRY(ptr(y, "y", T > 0));
    KDA_TRY(ptr(sfinal, "final_state", false));
    ConvParams p = conv_params(cfg);
    // strips of a document run at the same time and read the rows before their own
    const size_t state = conv_state(cfg, N);
    KDA_TRY(outputs_apart({{y, (size_t)T * cfg->C * elem(cfg->out_dtype), "y", 0}, {sfinal, state, "final_state", 0}},
                          {{x, extent(T, p.x_stride, p.C, elem(cfg->in_dtype)), "x", 0}, {weight, conv_weights(cfg), "weight", 0},
                           {bias, conv_bias(cfg), "bias", 0}, {cu, cu_bytes(N), "cu_seqlens", 0}, {s0, state, "initial_state", 0}}));
    int64_t slots;
    KDA_TRY(conv_plan(cfg, T, N, false, &p.len, &slots));
    p.x = x; p.weight = weight; p.bias = bias; p.cu = cu; p.s0 = s0; p.y = y; p.sfinal = sfinal;
    p.T = T; p.N = N; p.seqlen = cu ? 0 : (int32_t)(T / N); p.slots = (int32_t)slots; p.eight = conv_eight(cfg, T);
    return launched(launch_conv_fwd(p, cfg->width, cfg->in_dtype == KDA_BF16, (hipStream_t)stream));
}

size_t kda_conv_bwd_workspace_size(const kda_conv_config* cfg, int64_t T, int32_t N) {
    int32_t len;
    int64_t slots;
    if (check_conv(cfg) != KDA_OK || check_sizes(T, N) != KDA_OK || conv_plan(cfg, T, N, true, &len, &slots) != KDA_OK) return 0;
    return (size_t)slots * (cfg->width + 1) * cfg->C * sizeof(float);
}

kda_status kda_conv_bwd(const kda_conv_config* cfg, int64_t T, int32_t N, const void* x, const void* weight, const void* bias,
                        const int32_t* cu, const void* s0, const void* dy, const void* dsf, void* dx, float* dw, float* db,
                        void* ds0, void* workspace, size_t workspace_bytes, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_conv(cfg));
    KDA_TRY(check_sizes(T, N));
    KDA_TRY(check_stream(T, N, cu));
    KDA_TRY(ptr(x, "x", T > 0));
    KDA_TRY(ptr(weight, "weight", true));
    KDA_TRY(ptr(bias, "bias", false));
    KDA_TRY(ptr(s0, "initial_state", false));
    KDA_TRY(ptr(dy, "dy", T > 0));
    KDA_TRY(ptr(dsf, "d_final_state", false));
    KDA_TRY(ptr(dx, "dx", T > 0));
    KDA_TRY(ptr(dw, "dweight", true));
    KDA_TRY(ptr(db, "dbias", false));
    KDA_TRY(ptr(ds0, "d_initial_state", false));
    ConvParams p = conv_params(cfg);
    const size_t es = elem(cfg->in_dtype), state = conv_state(cfg, N), rows = (size_t)T * cfg->C;
    KDA_TRY(outputs_apart({{dx, rows * elem(cfg->out_dtype), "dx", 0}, {dw, (size_t)cfg->C * cfg->width * sizeof(float), "dweight", 0},
                           {db, cfg->C * sizeof(float), "dbias", 0}, {ds0, state, "d_initial_state", 0}},
                          {{x, extent(T, p.x_stride, p.C, es), "x", 0}, {weight, conv_weights(cfg), "weight", 0},
                           {bias, conv_bias(cfg), "bias", 0}, {cu, cu_bytes(N), "cu_seqlens", 0}, {s0, state, "initial_state", 0},
                           {dy, rows * es, "dy", 0}, {dsf, state, "d_final_state", 0}}));
    int64_t slots;
    KDA_TRY(conv_plan(cfg, T, N, true, &p.len, &slots));
    const size_t need = kda_conv_bwd_workspace_size(cfg, T, N);
    if (workspace_bytes < need) return fail(KDA_ERR_WORKSPACE, "workspace too small%s");
    KDA_TRY(ptr(workspace, "workspace", true));
    p.x = x; p.weight = weight; p.bias = bias; p.cu = cu; p.s0 = s0; p.dy = dy; p.dsf = dsf; p.dx = dx; p.ds0 = ds0;
    p.part = (float*)workspace;
    p.T = T; p.N = N; p.seqlen = cu ? 0 : (int32_t)(T / N); p.slots = (int32_t)slots; p.eight = conv_eight(cfg, T);
    return launched(launch_conv_bwd(p, cfg->width, cfg->in_dtype == KDA_BF16, dw, db, (hipStream_t)stream));
}

kda_status kda_conv_decode(const kda_conv_config* cfg, int32_t N, const void* x, const void* weight, const void* bias,
                           const void* state_in, void* state_out, void* y, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_conv(cfg));
    if (N < 0) return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 0%s");
    if (!grid_fits(((int64_t)N * cfg->C + kLayerThreads - 1) / kLayerThreads, kLayerThreads))
        return fail(KDA_ERR_UNSUPPORTED, "num_seqs * C too large for one launch%s");
    KDA_TRY(ptr(x, "x", N > 0));
    KDA_TRY(ptr(weight, "weight", N > 0));
    KDA_TRY(ptr(bias, "bias", false));
    KDA_TRY(ptr(state_in, "state_in", false));
    KDA_TRY(ptr(state_out, "state_out", N > 0));
    KDA_TRY(ptr(y, "y", N > 0));
    ConvParams p = conv_params(cfg);
    const size_t state = conv_state(cfg, N);
    if (state_in != state_out && overlap(state_in, state, state_out, state))
        return fail(KDA_ERR_INVALID_ARG, "state_in and state_out overlap without being equal%s");
    // a thread reads its channels before it writes them
    KDA_TRY(outputs_apart({{y, (size_t)N * cfg->C * elem(cfg->out_dtype), "y", cfg->out_dtype == cfg->in_dtype ? kRowsOf : 0},
                           {state_out, state, "state_out", kStates}},
                          {{x, extent(N, p.x_stride, p.C, elem(cfg->in_dtype)), "x", kRowsOf}, {weight, conv_weights(cfg), "weight", 0},
                           {bias, conv_bias(cfg), "bias", 0}, {state_in, state, "state_in", kStates}}));
    if (N == 0) return KDA_OK;
    p.x = x; p.weight = weight; p.bias = bias; p.s0 = state_in; p.sfinal = state_out; p.y = y; p.N = N;
    return launched(launch_conv_decode(p, cfg->width, cfg->in_dtype == KDA_BF16, (hipStream_t)stream));
}

void kda_selective_config_init(kda_selective_config* cfg, int32_t C, int32_t S, int32_t G) {
    if (!cfg) return;
    memset(cfg, 0, sizeof *cfg);
    cfg->C = C; cfg->S = S; cfg->G = G;
    cfg->flags = KDA_SELECTIVE_SOFTPLUS;
}

size_t kda_selective_fwd_workspace_size(const kda_selective_config* cfg, int64_t T, int32_t N) {
    if (check_selective(cfg) != KDA_OK || check_selective_sizes(cfg, T, N) != KDA_OK) return 0;
    return selective_plan(cfg, T, N, false).total;
}
size_t kda_selective_bwd_workspace_size(const kda_selective_config* cfg, int64_t T, int32_t N) {
    if (check_selective(cfg) != KDA_OK || check_selective_sizes(cfg, T, N) != KDA_OK) return 0;
    return selective_plan(cfg, T, N, true).total;
}

static kda_status check_selective_call(const kda_selective_config* cfg, int64_t T, int32_t N, const void* x, const void* dt,
                                       const float* A, const void* B, const void* C, const float* D, const void* z,
                                       const float* bias, const int32_t* cu, const float* s0) {
    KDA_TRY(check_selective(cfg));
    KDA_TRY(check_selective_sizes(cfg, T, N));
    KDA_TRY(check_stream(T, N, cu));
    KDA_TRY(ptr(x, "x", T > 0));
    KDA_TRY(ptr(dt, "dt", T > 0));
    KDA_TRY(ptr(A, "A", true));
    KDA_TRY(ptr(B, "B", T > 0));
    KDA_TRY(ptr(C, "C", T > 0));
    KDA_TRY(ptr(D, "D", false));
    KDA_TRY(ptr(z, "z", false));
    KDA_TRY(ptr(bias, "dt_bias", false));
    return ptr(s0, "initial_state", false);
}

kda_status kda_selective_fwd(const kda_selective_config* cfg, int64_t T, int32_t N, const void* x, const void* dt, const float* A,
                             const void* B, const void* C, const float* D, const void* z, const float* bias, const int32_t* cu,
                             const float* s0, void* y, float* sfinal, void* workspace, size_t workspace_bytes, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_selective_call(cfg, T, N, x, dt, A, B, C, D, z, bias, cu, s0));
    KDA_TRY(ptr(y, "y", T > 0));
    KDA_TRY(ptr(sfinal, "final_state", false));
    const SelectiveSizes n(cfg, T, N);
    // a lane has its own channel's rows of a block of tokens before it writes any of them
    KDA_TRY(outputs_apart({{y, n.out, "y", n.in_place}, {sfinal, n.state, "final_state", 0}},
                          {{x, n.x, "x", kRowsOf}, {dt, n.dt, "dt", kRowsOf}, {z, n.z, "z", kRowsOf}, {A, n.A, "A", 0}, {B, n.B, "B", 0},
                           {C, n.C, "C", 0}, {D, n.D, "D", 0}, {bias, n.D, "dt_bias", 0}, {cu, cu_bytes(N), "cu_seqlens", 0},
                           {s0, n.state, "initial_state", 0}}));
    const SelectivePlan f = selective_plan(cfg, T, N, false);
    if (workspace_bytes < f.total) return fail(KDA_ERR_WORKSPACE, "workspace too small%s");
    KDA_TRY(ptr(workspace, "workspace", f.total > 0));
    SelectiveParams p = selective_params(cfg);
    p.x = x; p.dt = dt; p.A = A; p.B = B; p.Cm = C; p.D = D; p.z = z; p.bias = bias; p.cu = cu; p.s0 = s0; p.y = y; p.sfinal = sfinal;
    p.T = T; p.N = N; p.seqlen = cu ? 0 : (int32_t)(T / N); p.len = (int32_t)f.len; p.slots = (int32_t)f.slots; p.cut = f.cut;
    char* ws = (char*)workspace;
    const int in = cfg->in_dtype == KDA_BF16;
    if (f.cut) {
        p.seg = (float*)(ws + f.seg);
        p.sdt = (float*)(ws + f.sdt);
        KDA_TRY(launched(launch_selective_states(p, cfg->S, in, false, (hipStream_t)stream)));
    }
    return launched(launch_selective_out(p, cfg->S, in, (hipStream_t)stream));
}

kda_status kda_selective_bwd(const kda_selective_config* cfg, int64_t T, int32_t N, const void* x, const void* dt, const float* A,
                             const void* B, const void* C, const float* D, const void* z, const float* bias, const int32_t* cu,
                             const float* s0, const void* dy, const float* dsf, void* dx, void* ddt, float* dA, void* dB, void* dC,
                             float* dD, void* dz, float* dbias, float* ds0, void* workspace, size_t workspace_bytes, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_selective_call(cfg, T, N, x, dt, A, B, C, D, z, bias, cu, s0));
    KDA_TRY(ptr(dy, "dy", T > 0));
    KDA_TRY(ptr(dsf, "dS_final", false));
    KDA_TRY(ptr(dx, "dx", T > 0));
    KDA_TRY(ptr(ddt, "ddt", T > 0));
    KDA_TRY(ptr(dA, "dA", true));
    KDA_TRY(ptr(dB, "dB", T > 0));
    KDA_TRY(ptr(dC, "dC", T > 0));
    KDA_TRY(ptr(dD, "dD", false));
    KDA_TRY(ptr(dz, "dz", T > 0 && z));
    KDA_TRY(ptr(dbias, "ddt_bias", false));
    KDA_TRY(ptr(ds0, "d_initial_state", false));
    const SelectiveSizes n(cfg, T, N);
    // as in the forward; the walks that read the others' rows have ended before
    KDA_TRY(outputs_apart({{dx, n.out, "dx", n.in_place}, {ddt, n.out, "ddt", n.in_place}, {z ? dz : nullptr, n.out, "dz", n.in_place},
                           {dA, n.A, "dA", 0}, {dB, n.dB, "dB", 0}, {dC, n.dB, "dC", 0}, {dD, n.D, "dD", 0}, {dbias, n.D, "ddt_bias", 0},
                           {ds0, n.state, "d_initial_state", 0}},
                          {{x, n.x, "x", kRowsOf}, {dt, n.dt, "dt", kRowsOf}, {z, n.z, "z", kRowsOf}, {dy, n.dy, "dy", kRowsOf},
                           {A, n.A, "A", 0}, {B, n.B, "B", 0}, {C, n.C, "C", 0}, {D, n.D, "D", 0}, {bias, n.D, "dt_bias", 0},
                           {cu, cu_bytes(N), "cu_seqlens", 0}, {s0, n.state, "initial_state", 0}, {dsf, n.state, "dS_final", 0}}));
    const SelectivePlan f = selective_plan(cfg, T, N, true);
    if (workspace_bytes < f.total) return fail(KDA_ERR_WORKSPACE, "workspace too small%s");
    KDA_TRY(ptr(workspace, "workspace", true));
    SelectiveParams p = selective_params(cfg);
    p.x = x; p.dt = dt; p.A = A; p.B = B; p.Cm = C; p.D = D; p.z = z; p.bias = bias; p.cu = cu; p.s0 = s0;
    p.dy = dy; p.dsf = dsf; p.dx = dx; p.ddt = ddt; p.dA = dA; p.dB = dB; p.dC = dC; p.dD = dD; p.dz = dz; p.dbias = dbias; p.ds0 = ds0;
    p.T = T; p.N = N; p.seqlen = cu ? 0 : (int32_t)(T / N); p.len = (int32_t)f.len; p.slots = (int32_t)f.slots; p.cut = f.cut;
    char* ws = (char*)workspace;
    p.seg = (float*)(ws + f.seg); p.sdt = (float*)(ws + f.sdt); p.rseg = (float*)(ws + f.rseg);
    p.border = (float*)(ws + f.border); p.bdt = (float*)(ws + f.bdt);
    p.bc_part = (float*)(ws + f.bc); p.par_part = (float*)(ws + f.par);
    const int in = cfg->in_dtype == KDA_BF16;
    KDA_TRY(launched(launch_selective_states(p, cfg->S, in, true, (hipStream_t)stream)));
    return launched(launch_selective_grads(p, cfg->S, in, (hipStream_t)stream));
}

kda_status kda_selective_decode(const kda_selective_config* cfg, int32_t N, const void* x, const void* dt, const float* A,
                                const void* B, const void* C, const float* D, const void* z, const float* bias,
                                const float* state_in, float* state_out, void* y, void* stream) {
    error_text()[0] = 0;
    KDA_TRY(check_selective(cfg));
    if (N < 0) return fail(KDA_ERR_INVALID_ARG, "num_seqs must be >= 0%s");
    if (!grid_fits(((int64_t)N * cfg->C * (cfg->S / 4) + kLayerThreads - 1) / kLayerThreads, kLayerThreads))
        return fail(KDA_ERR_UNSUPPORTED, "num_seqs * C too large for one launch%s");
    KDA_TRY(ptr(x, "x", N > 0));
    KDA_TRY(ptr(dt, "dt", N > 0));
    KDA_TRY(ptr(A, "A", N > 0));
    KDA_TRY(ptr(B, "B", N > 0));
    KDA_TRY(ptr(C, "C", N > 0));
    KDA_TRY(ptr(D, "D", false));
    KDA_TRY(ptr(z, "z", false));
    KDA_TRY(ptr(bias, "dt_bias", false));
    KDA_TRY(ptr(state_in, "state_in", false));
    KDA_TRY(ptr(state_out, "state_out", N > 0));
    KDA_TRY(ptr(y, "y", N > 0));
    const SelectiveSizes n(cfg, N, N);
    if (state_in != state_out && overlap(state_in, n.state, state_out, n.state))
        return fail(KDA_ERR_INVALID_ARG, "state_in and state_out overlap without being equal%s");
    // the lanes that share a channel are in one wave and read its values before the first of them writes
    KDA_TRY(outputs_apart({{y, n.out, "y", n.in_place}, {state_out, n.state, "state_out", kStates}},
                          {{x, n.x, "x", kRowsOf}, {dt, n.dt, "dt", kRowsOf}, {z, n.z, "z", kRowsOf}, {A, n.A, "A", 0}, {B, n.B, "B", 0},
                           {C, n.C, "C", 0}, {D, n.D, "D", 0}, {bias, n.D, "dt_bias", 0}, {state_in, n.state, "state_in", kStates}}));
    if (N == 0) return KDA_OK;
    SelectiveParams p = selective_params(cfg);
    p.x = x; p.dt = dt; p.A = A; p.B = B; p.Cm = C; p.D = D; p.z = z; p.bias = bias; p.s0 = state_in; p.sfinal = state_out; p.y = y;
    p.N = N;
    return launched(launch_selective_decode(p, cfg->S, cfg->in_dtype == KDA_BF16, (hipStream_t)stream));
}

}  // extern "C"
