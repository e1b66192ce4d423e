// dn_gated_scan.h -- what the C-ABI layer and the kernels of the gated linear
// recurrence (dn_gated_scan_plan.cpp, dn_gated_scan.hip) share.  Layouts as in include/dn.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace dn {

constexpr int kGsSaved = 128;   // steps between two saved states

struct GsProblem {
    int B, H, T, d;
    int bf16, coupled;
};
struct GsFwd {
    const void* x;
    const float* g;
    const int* lens;
    const float* h0;
    void* o;
    float* hT;
    float* states;
    int first_tile = 0;   // a chain begins with it; not 0 in tests alone, where the messages of those before it never come
};
struct GsBwd {
    const void* x;
    const float* g;
    const int* lens;
    const float* h0;
    const void* dout;
    const float* dhT;
    const float* states;   // NULL: recomputed in the workspace
    void* dx;
    float *dg, *dh0;
    int first_tile = 0;
};
size_t gs_states_bytes(const GsProblem& pr);
// pass: 0 forward, 1 backward with saved states, 2 backward recomputing them
size_t gs_workspace_bytes(const GsProblem& pr, int pass);
// strips of 64 channels: whether one launch holds them
bool gs_fits(const GsProblem& pr);
hipError_t launch_gated_scan_fwd(const GsProblem& pr, const GsFwd& f, char* ws, hipStream_t s);
hipError_t launch_gated_scan_bwd(const GsProblem& pr, const GsBwd& f, char* ws, hipStream_t s);
hipError_t launch_gated_scan_recurrent(const GsProblem& pr, const void* x, const float* g, float* state, void* o,
                                       hipStream_t s);

}  // namespace dn
