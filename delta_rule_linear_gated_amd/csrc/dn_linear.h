// dn_linear.h -- what the host side and the kernels of linear attention with a
// decay per head share: the arguments of a launch and the split of the steps.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dn {

enum LinGate { kLinNone = 0, kLinScalar = 1, kLinHead = 2 };

constexpr int kLinC = 64;         // steps of a chunk
constexpr int kLinSnap = 16;      // chunks between kept states, for the gate gradient

// One evaluation of
//     out_i = sum_{j <= i} w_ij (x_i . y_j) z_j + w_i (S0 x_i),
//     S_t = e^{g_t} S_{t-1} + z_t y_t^T      (rows over z's channels),
// over one (b, h), w_ij the decay between the steps.  rev: the steps run from the
// last to the first and a step's gate is the one after it (the cotangent of the
// state: D_t = z_t y_t^T + e^{g_{t+1}} D_{t+1}).
//   forward output  (x, y, z) = (q, k, v)     dv  = (k, q, dout), rev
//   dq              = (dout, v, k)            dk  = (v, dout, q), rev
struct LinOp {
    const void* x;
    const void* y;
    const void* z;
    void* out;
    const float* init;   // state before the first step (NULL: zero)
    float* fin;          // state after the last one (NULL: not wanted)
    float* snap;         // kept states [BH][nent + 1][dv][dk] (see LinArgs)
    long snap_bh;        // floats of one (b, h) there
    int sn, sk;          // strides of state element (z channel, y channel) in init, fin, snap
    int rev;
    // Gate gradient: rows r laid out like z; dots[2][blk][BH][T] = r_i . out_i, over the block's
    // channels and before its rounding: the part from earlier chunks, then from all steps before
    const void* r;
    float* dots;
};

// State entries: forward, entry e = the state before chunk e * snap; rev, entry e = the
// state that enters chunks [e * snap, (e + 1) * snap) from the right; entry nent = the
// last state of the evaluation.  Parallel segments cover seg_len chunks (a multiple of
// snap).
struct LinArgs {
    LinOp op[3];
    int nops, BH, H, T, NT;
    int kd, nd, nblk;    // channels of x and y, of z and out; blocks of z channels
    int nseg, seg_len, snap, nent;
    const float* g;
    int gate;            // LinGate
    const int* lens;     // [B] or NULL
    float* segdec;       // [nops][BH][nseg] decay factor of each parallel segment
};

// Split of the steps for BH heads: nseg parallel segments, kept states every snap chunks.
struct LinPlan {
    int nseg, seg_len, snap, nent;
};

// z channels of one workgroup: registers hold that many state rows.
__host__ __device__ constexpr int lin_vb(int nd, bool bf16) {
    return nd < (bf16 ? 64 : 32) ? nd : (bf16 ? 64 : 32);
}

// Lengths are data on the device: clamped to [0, T] here.
__device__ __forceinline__ int lin_len(const int* lens, int b, int T) {
    if (!lens) return T;
    const int n = lens[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

enum LinMode { kLinState = 0, kLinOut = 1, kLinDots = 2 };
// Output tiles (16 channels) whose 16-byte pieces a lane stores at once.
__host__ __device__ constexpr int lin_pair(bool bf16, int nv) { return bf16 && nv > 1 ? 2 : 1; }
// The gate's gradient leaves room for one workgroup on a compute unit (three parts of the
// state in LDS): eight waves form its outputs, each half of the channels, so that matrix,
// vector and LDS work of more waves overlap (8 x 16 heads, 4096 steps, when it was chosen:
// 580 us, four waves 607, and 1010 in 128 registers with two workgroups on a unit, which
// spill; 512 now).  The outputs alone, at 128 x 64 channels, are faster on four (163 us against
// 190, ragged prompts of 8 x 16 heads).
__host__ __device__ constexpr int lin_halves(int mode, bool bf16, int nv) {
    return mode == kLinDots && nv / lin_pair(bf16, nv) > 1 ? 2 : 1;
}
// Four waves carry the state; four for each share of the channels form the outputs.
__host__ __device__ constexpr int lin_threads(int mode, bool bf16, int nv) {
    return mode == kLinState ? 256 : 256 + 256 * lin_halves(mode, bf16, nv);
}
// Waves a SIMD holds at once: the registers of fp32 rows and of the gate's gradient leave
// room for few, LDS at 128 x 64 channels for one workgroup.
__host__ __device__ constexpr int lin_waves(int mode, bool bf16, int kd, int nv) {
    return mode == kLinOut && bf16 && kd * nv < 128 * 4 ? 4 : 2;
}
typedef hipError_t (*LinLaunch)(const LinArgs& a, int nv, int mode, hipStream_t s);
hipError_t lin_bf16_k32(const LinArgs&, int, int, hipStream_t);
hipError_t lin_bf16_k64(const LinArgs&, int, int, hipStream_t);
hipError_t lin_bf16_k128(const LinArgs&, int, int, hipStream_t);
hipError_t lin_f32_k32(const LinArgs&, int, int, hipStream_t);
hipError_t lin_f32_k64(const LinArgs&, int, int, hipStream_t);
hipError_t lin_f32_k128(const LinArgs&, int, int, hipStream_t);

}  // namespace dn
