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
constexpr int kSegDocs = 512;     // more documents than this are not cut into segments
constexpr int kGradThreads = 512; // 8 wave64: one 16-row block of a 128-token block each

// g[token * g_stride + head]: g_stride = H for a gate per token, 0 for a gate per head.
// seg_len: 0 for one walk per document, else tokens per segment (a multiple of kLinBlock).
// chains: (document or segment slot, head) pairs.
struct LinearParams {
    const void* q;         // [T,Hk,dk]
    const void* k;         // [T,Hk,dk]
    const void* v;         // [T,H,dv]
    const float* g;
    const int32_t* cu;     // device [N+1] or nullptr (equal documents of `seqlen`)
    const float* s0;       // [N,H,dk,dv] or nullptr (zero)
    const float* seg_state; // [slots,H,dk,dv]: the states entering the segments after a document's first
    void* o;               // [T,H,dv] out dtype
    float* sfinal;         // [N,H,dk,dv] or nullptr
    int64_t T;
    int32_t N, H, Hk, dv, seqlen, g_stride, seg_len, out_bf16, chains, longest_first;
    float scale;
};

// A walk that only carries the state, forward (a = k, b = v) or in reverse (a = q, b = dO).
// With `decay` it starts from zero and leaves the segment's own sum in `seg`; without, it
// starts from s0 or the carried `seg`.
struct LinearStateDir {
    const void* a;         // [T,Hk,dk]
    const void* b;         // [T,H,dv]
    const float* s0;       // [N,H,dk,dv] or nullptr (zero)
    float* seg;            // [slots,H,dk,dv]
    float* decay;          // [slots,H] e^{sum of g} of the segment, or nullptr
    float* last;           // [N,H,dk,dv] or nullptr: the state after the document
    void* border;          // state before every 128-token block (input type) [blocks,H,dk,dv], or nullptr
    int32_t rev;
};
struct LinearStateParams {
    LinearStateDir dir[2];
    const float* g;
    const int32_t* cu;
    int64_t T;
    int32_t N, H, Hk, dv, seqlen, g_stride, seg_len, whole_len, chains, dirs;   // whole_len: see segment_length
    float scale;
};

// From the segments' own sums to the states entering them, in place.
struct LinearCarryDir {
    const float* s0;       // [N,H,dk,dv] or nullptr
    float* seg;            // [slots,H,dk,dv]
    const float* decay;    // [slots,H]
    int32_t rev;
};
struct LinearCarryParams {
    LinearCarryDir dir[2];
    const int32_t* cu;
    int64_t T;
    int32_t N, H, seqlen, seg_len, whole_len, elems, slots;   // elems = dk * dv; slots: room for segments
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
    float* sums;           // [2][parts,T,Hk,dk] dq and dk summed over a part's value heads (parts > 1)
    float* dg_part;        // [blocks,H] sum of dg over the block (gate per head), or nullptr
    void* dq;
    void* dk_out;
    void* dv_out;
    void* dg;
    int64_t T, blocks;
    int32_t N, H, Hk, dv, seqlen, g_stride, out_bf16, dg_bf16, parts;   // parts divides H / Hk
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

// At most so many pieces of `piece` tokens in the documents of a stream.
inline int64_t linear_slots(int64_t T, int32_t N, int32_t piece) { return T / piece + N; }

hipError_t launch_linear_out(const LinearParams& p, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_linear_states(const LinearStateParams& p, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_linear_carry(const LinearCarryParams& p, int dirs, hipStream_t stream);
hipError_t launch_linear_grads(const LinearBwdParams& p, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_linear_decode(const LinearDecodeParams& p, int in_dtype, int dk, hipStream_t stream);

}  // namespace kda
