// dn_qk.h -- what the C-ABI layer and the kernels of the queries' and keys' norms and
// rotations (dn_qk_plan.cpp, dn_qk.hip, dn_qk_kernels.h) share.  Layouts as in include/dn.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace dn {

enum QkTurn { kTurnNone = 0, kTurnHalves = 1, kTurnNeighbours = 2 };

// One of q and k: rows [B][heads][T][d], those of x and out by strides in elements.
struct QkSide {
    int heads;
    const void *x, *dy;          // dy: dense (backward of a norm)
    const float* w;              // [d] or NULL
    void* out;                   // y or dx
    float* dw;                   // [d] or NULL
    long xs[3], os[3];           // batch, head, step of x and of out
};
struct QkArgs {
    int B, T, d, rot;
    int bf16, turn, back;        // back: angles negated (the gradient of a rotation)
    int norm;                    // 0 none, 1 by the row's length, 2 by its root mean square
    float eps, share, amplitude; // share: of the sum of squares (1 or 1 / d)
    const double* freqs;
    const int *pos, *lens;
    int pos_kind;                // 0: t, 1: pos[b] + t, 2: pos[b][t]
    QkSide side[2];
    float* parts;                // partial sums of dw
    int tiles, groups[2], per;   // launch: workgroups of a head group, head groups of each side, heads of a group
};
void qk_split(QkArgs* a, bool bwd);
bool qk_fits(const QkArgs& a);   // whether one launch holds it
size_t qk_workspace_bytes(const QkArgs& a);
hipError_t launch_qk_fwd(QkArgs a, hipStream_t s);
hipError_t launch_qk_bwd(QkArgs a, char* ws, hipStream_t s);

typedef hipError_t (*QkLaunch)(const QkArgs&, unsigned blocks, hipStream_t);
hipError_t qk_fwd_bf16(const QkArgs&, unsigned, hipStream_t);
hipError_t qk_fwd_f32(const QkArgs&, unsigned, hipStream_t);
hipError_t qk_bwd_bf16(const QkArgs&, unsigned, hipStream_t);
hipError_t qk_bwd_f32(const QkArgs&, unsigned, hipStream_t);

}  // namespace dn
