// dn_tree.h -- what the C-ABI layer and the kernels of drafted-token trees share.
// Layouts as in include/dn.h.
#pragma once

#include <hip/hip_runtime.h>

namespace dn {

constexpr int kTreeMax = 64;   // nodes of a tree: one lane each

struct TreeArgs {
    int B, H, N, dk, dv;
    int bf16;
    int gate;            // dn_gate
    int kz;              // beta holds eta
    float eps;
    const void *q, *k, *v;
    const float *beta;   // NULL: linear attention
    const float *g;
    const int *parent;   // [B][N]
    const int *counts;   // [B] or NULL
    const int *accept;   // [B] (commit)
    float* state;
    void* o;
    float* u;            // written by fwd (or NULL), read by commit
};

hipError_t launch_tree_fwd(const TreeArgs& a, hipStream_t s);
hipError_t launch_tree_commit(const TreeArgs& a, hipStream_t s);

typedef hipError_t (*TreeLaunch)(const TreeArgs&, hipStream_t);
hipError_t tree_fwd_bf16(const TreeArgs&, hipStream_t);
hipError_t tree_fwd_f32(const TreeArgs&, hipStream_t);

}  // namespace dn
