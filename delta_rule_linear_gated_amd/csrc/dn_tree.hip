// dn_tree.hip -- launches of the drafted-token operators and the commit of an accepted
// path into the state.
#include "dn_internal.h"
#include "dn_tree_kernels.h"

namespace dn {

namespace {

// The state moved along the accepted path a:
//     S <- S e^{Gam_a} + sum_{m on the path} u_m (k_m e^{Gam_a - Gam_m})^T,
// in place.  A workgroup takes one (b, h) and 64 state rows, 16 lanes a row (as the
// recurrent kernels: whole cache lines of the state, which is nearly all the bytes), the
// path's keys (decayed to its end) and u rows in LDS, loaded while the state's rows are
// on their way.  A sequence that accepts nothing is neither read nor written.
constexpr int kCommitThreads = 256, kCommitRows = 64;

template <typename T, int DK, int NP>
__global__ __launch_bounds__(kCommitThreads) void tree_commit_kernel(TreeArgs a) {
    constexpr int E = DK / 16, R = kCommitRows / 16, LU = kCommitRows + 4;
    __shared__ __align__(16) float kd[NP][DK];
    __shared__ __align__(16) float us[NP][LU];
    __shared__ float end[DK];       // e^{Gam_a} of each channel
    __shared__ float wt[NP];        // e^{Gam_a - Gam_m} of a gate per step or head
    __shared__ int path[NP];        // the path, root first
    const int nblk = (a.dv + kCommitRows - 1) / kCommitRows;
    int bh, blk;
    head_and_block(nblk, a.B * a.H, bh, blk);
    const int b = bh / a.H, h = bh % a.H, N = a.N, tid = threadIdx.x, l = lane_id(), j = l & 15;
    const int at = __builtin_amdgcn_readfirstlane(a.accept[b]);
    const int cnt = a.counts ? __builtin_amdgcn_readfirstlane(a.counts[b]) : N;
    if (at < 0 || at >= min(cnt, N)) return;
    const long rows = (long)bh * N;

    // ---- the tree's loads, then state rows r = 16 i + tid / 16 of the block
    const int p = tree_parent(a.parent + (long)b * N, N, l);
    double x = 0.0;
    if (l < N && a.gate == DN_GATE_SCALAR) x = tree_clamp(a.g[rows + l]);
    if (l < N && a.gate == DN_GATE_HEAD) x = tree_clamp(a.g[h]);
    float s[R][E];
    float* base = a.state + ((long)bh * a.dv + blk * kCommitRows) * DK + j * E;
    const int left = a.dv - blk * kCommitRows;   // rows of the block
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = min(16 * i + (tid >> 4), left - 1);
#pragma unroll
        for (int e = 0; e < E; ++e) s[i][e] = base[(long)r * DK + e];
    }

    // ---- the path (every wave for itself; wave 0 writes it down)
    const unsigned long long all = tree_path<NP>(p, l, x);
    const unsigned long long on = __shfl(all, at);
    const double xe = __shfl(x, at);
    const int len = __popcll(on);
    if (tid < 64 && (on >> l & 1)) {
        const int i = __popcll(on & ((1ull << l) - 1));
        path[i] = l;
        wt[i] = expf((float)(xe - x));
    }
    __syncthreads();
    if (a.gate == DN_GATE_VECTOR) {   // from the path's end up, a channel a thread, sums of its gates
        for (int c = tid; c < DK; c += kCommitThreads) {
            float w = 0.f;
            for (int i = len - 1; i >= 0; --i) {
                kd[i][c] = expf(w);
                w += tree_clamp(a.g[(rows + path[i]) * DK + c]);
            }
            end[c] = expf(w);
        }
        __syncthreads();
    }
    for (int id = tid; id < len * DK; id += kCommitThreads) {
        const int i = id / DK, c = id % DK;
        const float w = a.gate == DN_GATE_VECTOR ? kd[i][c] : wt[i];
        kd[i][c] = to_f(static_cast<const T*>(a.k)[(rows + path[i]) * DK + c]) * w;
    }
    for (int id = tid; id < len * kCommitRows; id += kCommitThreads) {
        const int i = id / kCommitRows, r = id % kCommitRows;
        us[i][r] = r < left ? a.u[(rows + path[i]) * a.dv + blk * kCommitRows + r] : 0.f;
    }
    const float e1 = a.gate == DN_GATE_VECTOR ? 1.f : expf((float)xe);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float w = a.gate == DN_GATE_VECTOR ? end[j * E + e] : e1;
#pragma unroll
        for (int i = 0; i < R; ++i) s[i][e] *= w;
    }
    for (int q = 0; q < len; ++q) {
        float kk[E];
#pragma unroll
        for (int e = 0; e < E; ++e) kk[e] = kd[q][j * E + e];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float u = us[q][16 * i + (tid >> 4)];
#pragma unroll
            for (int e = 0; e < E; ++e) s[i][e] += u * kk[e];
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = 16 * i + (tid >> 4);
        if (r < left) {
#pragma unroll
            for (int e = 0; e < E; ++e) base[(long)r * DK + e] = s[i][e];
        }
    }
}

template <typename T, int DK> hipError_t commit_dk(const TreeArgs& a, hipStream_t s) {
    const int nblk = (a.dv + kCommitRows - 1) / kCommitRows;
    const dim3 grid((unsigned)((long)a.B * a.H * nblk)), block(kCommitThreads);
    // LDS for 64 nodes leaves three workgroups on a compute unit, for 16 nodes eight
    if (a.N <= 16)
        hipLaunchKernelGGL((tree_commit_kernel<T, DK, 16>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((tree_commit_kernel<T, DK, kTreeMax>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <typename T> hipError_t commit_launch(const TreeArgs& a, hipStream_t s) {
    switch (a.dk) {
        case 16: return commit_dk<T, 16>(a, s);
        case 32: return commit_dk<T, 32>(a, s);
        case 64: return commit_dk<T, 64>(a, s);
        case 128: return commit_dk<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_tree_fwd(const TreeArgs& a, hipStream_t s) {
    if ((long)a.B * a.H * a.N == 0) return hipSuccess;
    prof_begin(s, "tree_fwd");
    const hipError_t e = a.bf16 ? tree_fwd_bf16(a, s) : tree_fwd_f32(a, s);
    prof_end(s);
    return e;
}

hipError_t launch_tree_commit(const TreeArgs& a, hipStream_t s) {
    if ((long)a.B * a.H * a.N == 0) return hipSuccess;
    prof_begin(s, "tree_commit");
    const hipError_t e = a.bf16 ? commit_launch<bf16>(a, s) : commit_launch<float>(a, s);
    prof_end(s);
    return e;
}

}  // namespace dn
