// dn_qk.hip -- launches of the queries' and keys' norms and rotations
// (dn_qk_kernels.h): the split of tokens and heads, and the sums of the weights' gradients.
#include <algorithm>

#include "dn_device.h"
#include "dn_internal.h"
#include "dn_qk.h"

namespace dn {

namespace {

constexpr int kQkUnits = 256;   // compute units

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

// Heads a lane takes, and the workgroups.  More heads a lane share its angles; fewer fill the
// chip.  Measured at 32 + 32 heads of 128, 32768 steps, bf16 (us, rms with halves rotated, 4 / 8 /
// 16 heads): 234 / 223 / 217, backward without weights 347 / 329 / 328, with few tokens (16 + 16
// heads, 1024 steps) 7.5 / 8.0 / 7.3.
// As many workgroups as run at once, each walking the token tiles, keep reads and writes apart
// less than a workgroup a tile does: 4 a unit against 8 (backward, l2) 305 -> 350 us (6: 311, 3: 299,
// 2: 343), against one a tile (forward, l2) 211 -> 220, rotation alone 212 -> 221.  But the rotation
// back, whose rows lie head by head on both sides, takes 231 -> 217, and with the lengths of a
// padded batch the tiles differ in work (8 sequences of up to 4096 steps, 16 + 16 heads, forward:
// 101 -> 85): then a workgroup a tile, or in the backward, whose workgroups each leave a partial
// sum, 8 a unit.
void qk_split(QkArgs* a, bool bwd) {
    const long tokens = (long)a->B * a->T, per_wg = 256 / (a->d / 8);
    const long tiles = (tokens + per_wg - 1) / per_wg;
    const int most = std::max(a->side[0].heads, a->side[1].heads);
    int per = 8;
    auto groups = [&](int side) { return (a->side[side].heads + per - 1) / per; };
    while (per > 1 && (per >= 2 * most || tiles * (groups(0) + groups(1)) < 4 * kQkUnits)) per /= 2;
    a->per = per;
    a->groups[0] = groups(0);
    a->groups[1] = groups(1);
    const long all = std::max((long)a->groups[0] + a->groups[1], 1L);
    const bool uneven = a->lens || a->back;
    a->tiles = (int)(uneven && !bwd ? tiles : std::min<long>(tiles, std::max((uneven ? 8 : 4) * kQkUnits / all, 1L)));
}

}  // namespace

bool qk_fits(const QkArgs& in) {
    QkArgs a = in;
    a.back = 1;   // the most workgroups
    qk_split(&a, false);
    return (long)a.tiles * ((long)a.groups[0] + a.groups[1]) < (1L << 32) / 256;
}

size_t qk_workspace_bytes(const QkArgs& in) {
    QkArgs a = in;
    if ((long)a.B * a.T == 0) return 0;
    a.back = 1;   // the most workgroups, as with lengths
    qk_split(&a, true);
    return (size_t)a.tiles * (a.groups[0] + a.groups[1]) * a.d * 4;
}

hipError_t launch_qk_fwd(QkArgs a, hipStream_t s) {
    if ((long)a.B * a.T * (a.side[0].heads + a.side[1].heads) == 0) return hipSuccess;
    qk_split(&a, false);
    prof_begin(s, "qk_fwd");
    const hipError_t e = (a.bf16 ? qk_fwd_bf16 : qk_fwd_f32)(a, (unsigned)(a.tiles * (a.groups[0] + a.groups[1])), s);
    prof_end(s);
    return e;
}

hipError_t launch_qk_bwd(QkArgs a, char* ws, hipStream_t s) {
    const bool none = (long)a.B * a.T * (a.side[0].heads + a.side[1].heads) == 0;
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
