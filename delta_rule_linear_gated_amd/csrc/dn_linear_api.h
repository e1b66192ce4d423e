// dn_linear_api.h -- what the C-ABI layer calls for linear attention with a decay
// per head (dn_linear.hip).  Layouts as in include/dn.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace dn {

struct LinProblem {
    int B, H, T, dk, dv;
    int bf16, gate;   // gate: LinGate (0 none, 1 per step, 2 per head)
    int no_scan;      // one run of the steps per head, never parallel segments
};
struct LinFwd {
    const void *q, *k, *v;
    const float* g;
    const int* lens;
    const float* h0;
    void* o;
    float* hT;
};
struct LinBwd {
    const void *q, *k, *v;
    const float* g;
    const int* lens;
    const float* h0;
    const void* dout;
    const float* dhT;
    void *dq, *dk, *dv;
    float *dg, *dh0;
};
// pass: 0 forward, 1 backward
size_t lin_workspace_bytes(const LinProblem& pr, int pass);
hipError_t launch_linear_fwd(const LinProblem& pr, const LinFwd& f, char* ws, hipStream_t s);
hipError_t launch_linear_bwd(const LinProblem& pr, const LinBwd& f, char* ws, hipStream_t s);
hipError_t launch_linear_recurrent(const LinProblem& pr, const void* q, const void* k, const void* v, const float* g,
                                   float* state, void* o, hipStream_t s);

}  // namespace dn
