// kda_tree.h -- host-side interface of the drafted-tree kernels.  Not installed.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kTreeMaxNodes = 64;   // ancestor sets are 64-bit masks

struct TreeParams {
    const void* q;          // [N,L,Hk,dk] (kda_tree only)
    const void* k;          // [N,L,Hk,dk]
    const void* v;          // [N,L,H,dv]
    const void* g;          // delta rule: [N,L,H,dk] input type; linear rule: fp32 [N,L,H] or [H]
    const void* beta;       // delta rule: [N,L,H]
    const int32_t* parent;  // [N,L]
    const int32_t* accept;  // [N] (kda_tree_commit only)
    const float* s_in;      // [N,H,dk,dv] or nullptr (zero state)
    float* s_out;           // [N,H,dk,dv] (kda_tree_commit only)
    void* o;                // [N,L,H,dv] (kda_tree only)
    int32_t N, H, Hk, L, dv, gate_head, out_bf16;
    float eps, scale;
};

hipError_t launch_tree(const TreeParams& p, bool delta, int in_dtype, int dk, hipStream_t stream);
hipError_t launch_tree_commit(const TreeParams& p, bool delta, int in_dtype, int dk, hipStream_t stream);

}  // namespace kda
