// dn_qk.hip -- launches of the queries' and keys' norms and rotations
// (dn_qk_kernels.h), split as dn_qk_plan.cpp says, and the sums of the weights' gradients.
#include "dn_device.h"
#include "dn_internal.h"
#include "dn_qk.h"

namespace dn {

namespace {

// Sum of the workgroups' partial dw: 16 channels a workgroup, 64 threads a channel over the
// entries, eight loads in flight each (the sums are a chain of latencies: 16 threads with one
// load in flight took 29 us for 1024 entries).
__global__ __launch_bounds__(1024) void qk_dw_kernel(QkArgs a) {
    __shared__ float part[64][17];
    const int blocks = a.d / 16, sd = blockIdx.x / blocks, j = blockIdx.x % blocks * 16 + threadIdx.x % 16;
    if (!a.side[sd].dw) return;
    const int r = threadIdx.x / 16;
    const long first = sd ? (long)a.groups[0] * a.tiles : 0, n = (long)a.groups[sd] * a.tiles;
    float sum = 0.f;
    constexpr int AHEAD = 8;
    for (long i0 = r; i0 < n; i0 += 64 * AHEAD) {
        float v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) v[i] = a.parts[(first + min(i0 + 64 * i, n - 1)) * a.d + j];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) sum += i0 + 64 * i < n ? v[i] : 0.f;
    }
    part[r][threadIdx.x % 16] = sum;
    __syncthreads();
    if (r) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) sum += part[i][threadIdx.x];
    a.side[sd].dw[j] = sum;
}

}  // namespace

hipError_t launch_qk_fwd(QkArgs a, hipStream_t s) {
    if ((long)a.B * a.T * ((long)a.side[0].heads + a.side[1].heads) == 0) return hipSuccess;
    qk_split(&a, false);
    prof_begin(s, "qk_fwd");
    const hipError_t e = (a.bf16 ? qk_fwd_bf16 : qk_fwd_f32)(a, (unsigned)(a.tiles * (a.groups[0] + a.groups[1])), s);
    prof_end(s);
    return e;
}

hipError_t launch_qk_bwd(QkArgs a, char* ws, hipStream_t s) {
    const bool none = (long)a.B * a.T * ((long)a.side[0].heads + a.side[1].heads) == 0;
    hipError_t e = hipSuccess;
    qk_split(&a, true);
    a.parts = reinterpret_cast<float*>(ws);
    if (none) {
        a.tiles = 0;   // sums of nothing
    } else {
        prof_begin(s, "qk_bwd");
        e = (a.bf16 ? qk_bwd_bf16 : qk_bwd_f32)(a, (unsigned)(a.tiles * (a.groups[0] + a.groups[1])), s);
        prof_end(s);
    }
    if (e != hipSuccess || !(a.side[0].dw || a.side[1].dw)) return e;
    prof_begin(s, "qk_dw");
    hipLaunchKernelGGL(qk_dw_kernel, dim3(2 * a.d / 16), dim3(1024), 0, s, a);
    prof_end(s);
    return hipGetLastError();
}

}  // namespace dn
