// kda_linear.h -- shared by the kernels of the linear rule (scalar decay per head):
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// Host-side parameter structs, then the device helpers.  Not installed.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int kLinChunk = 64;     // tokens per step of the walks over a document
constexpr int kLinBlock = 128;    // tokens per gradient workgroup; saved states sit at its borders
constexpr int kWalkTarget = 512;  // workgroups a walk aims for: two a compute unit
constexpr int kGradThreads = 512; // 8 wave64: one 16-row block of a 128-token block each

// g[token * g_stride + head]: g_stride = H for a gate per token, 0 for a gate per head.
struct LinearParams {
    const void* q;         // [T,Hk,dk]
    const void* k;         // [T,Hk,dk]
    const void* v;         // [T,H,dv]
    const float* g;
    const int32_t* cu;     // device [N+1] or nullptr (equal documents of `seqlen`)
    const float* s0;       // entering states: [N,H,dk,dv] per document, or per segment slot when seg_len > 0
    void* o;               // [T,H,dv] out dtype
    float* sfinal;         // [N,H,dk,dv] or nullptr
    int64_t T;
    int32_t N, H, Hk, dv, seqlen, g_stride;
    int32_t seg_len;       // 0: one walk per document; else tokens per segment (a multiple of kLinBlock)
    int32_t out_bf16;
    int32_t chains;        // (document or segment slot, head) pairs
    float scale;
};

// A walk that only carries the state, forward (a = k, b = v) or in reverse (a = q, b = dO).
struct LinearStateDir {
    const void* a;         // [T,Hk,dk]
    const void* b;         // [T,H,dv]
    const float* s0;       // entering states, as in LinearParams, or nullptr (zero)
    float* last;           // state after the walk: [N,H,dk,dv], or per slot with `decay`; or nullptr
    float* decay;          // [slots,H] e^{sum of g} of the segment, or nullptr
    void* border;          // state before every 128-token block (input type) [blocks,H,dk,dv], or nullptr
    int32_t rev;
};
struct LinearStateParams {
    LinearStateDir dir[2];
    const float* g;
    const int32_t* cu;
    int64_t T;
    int32_t N, H, Hk, dv, seqlen, g_stride, seg_len, chains;
    float scale;
};

// The states entering every segment, from the segments' own sums: state (in place) [slots,H,dk,dv].
struct LinearCarryDir {
    const float* s0;       // [N,H,dk,dv] or nullptr
    float* state;
    const float* decay;    // [slots,H]
    float* last;           // [N,H,dk,dv] or nullptr
    int32_t rev;
};
struct LinearCarryParams {
    LinearCarryDir dir[2];
    const int32_t* cu;
    int64_t T;
    int32_t N, H, seqlen, seg_len, elems;   // elems = dk * dv
};

struct LinearBwdParams {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const int32_t* cu;
    const void* dO;        // [T,H,dv]
    const void* S;         // state entering every block (input type) [blocks,H,dk,dv]
    const void* dS;        // dL/dS at the end of every block
    float* e;              // [H,T] q . dq through the entering state, plus row sums of A (see kda_linear_bwd.hip)
    float* a;              // [H,T] column sums of A
    float* f;              // [H,T] k . dk through dS
    float* cross;          // [blocks,H] e^{G} <S, dS>
    float* dg_part;        // [blocks,H] sum of dg over the block (gate per head), or nullptr
    void* dq;
    void* dk_out;
    void* dv_out;
    void* dg;
    int64_t T, blocks;
    int32_t N, H, Hk, dv, seqlen, g_stride, out_bf16;
    float scale;
};

struct LinearDecodeParams {
    const void* q;         // [N,Hk,dk]
    const void* k;
    const void* v;         // [N,H,dv]
    const float* g;        // [N,H] or [H]
    const float* s_in;     // [N,H,dk,dv] or nullptr
    float* s_out;
    void* o;               // [N,H,dv]
    int32_t N, H, Hk, dv, g_stride, out_bf16;
    float scale;
};

// slots of a stream cut into pieces of `piece` tokens per document (see slot_owner)
inline int64_t linear_slots(int64_t T, int32_t N, int32_t piece) { return T / piece + N; }

hipError_t launch_linear_out(const LinearParams& p, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_linear_states(const LinearStateParams& p, int dirs, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_linear_carry(const LinearCarryParams& p, int dirs, hipStream_t stream);
hipError_t launch_linear_grads(const LinearBwdParams& p, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_linear_decode(const LinearDecodeParams& p, int in_dtype, int dk, hipStream_t stream);

}  // namespace kda
