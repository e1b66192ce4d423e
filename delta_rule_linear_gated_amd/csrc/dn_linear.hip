// dn_linear.hip -- linear attention with a decay per head: the split of the steps,
// the launch sequences, the kernels between the chunk kernels (dn_linear_kernels.h)
// and the recurrent form.
#include <algorithm>

#include "dn_device.h"
#include "dn_internal.h"
#include "dn_linear.h"
#include "dn_linear_api.h"

namespace dn {

namespace {

constexpr int kLinMaxSeg = 64;   // parallel segments of a sequence
constexpr int kLinUnits = 256;   // compute units

// Boundary states of the parallel segments: entry s of snap holds segment s's own
// contribution (from a zero state) and gets the state the segment starts from,
//     start_{s+1} = dec_s start_s + end_s,
// walked first to last (rev: last to first).  A thread owns one element of one (b, h)
// state and loads all N >= nseg entries of it at once: the walk itself is short, and
// waiting for the entries batch by batch took most of the time (4 heads, 64 segments:
// 23 us in four batches, 13 us at once).
template <int N> __global__ __launch_bounds__(256) void lin_join_kernel(LinArgs a) {
    const int se = a.kd * a.nd;   // a multiple of 256
    const int per = se / 256, oi = blockIdx.y;
    const int bh = blockIdx.x / per, at = (blockIdx.x % per) * 256 + threadIdx.x;
    const LinOp& op = a.op[oi];
    float* base = op.snap + bh * op.snap_bh + at;
    // one factor a lane: loaded once, not waited for at every entry
    static_assert(N <= 64, "a factor of each segment in a lane");
    const float dec = a.segdec[((long)oi * a.BH + bh) * a.nseg + min(lane_id(), a.nseg - 1)];
    float cur = op.init ? op.init[(long)bh * se + at] : 0.f;
    const int r = a.seg_len / a.snap, last = (a.NT - 1) / a.snap;
    auto slot = [&](int i) {   // i-th segment walked -> its entry
        const int s = op.rev ? a.nseg - 1 - i : i;
        return base + (long)(op.rev ? min((s + 1) * r - 1, last) : s * r) * se;
    };
    float own[N];
#pragma unroll
    for (int i = 0; i < N; ++i) own[i] = *slot(min(i, a.nseg - 1));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i < a.nseg) *slot(i) = cur;   // the last segment's own part is nowhere formed, nor used
        cur = cur * __shfl(dec, op.rev ? a.nseg - 1 - i : i) + own[i];
    }
}

// Sums over runs of steps: a thread owns steps ta .. ta + 3 of [lo, hi), bit i of cuts says
// that a run starts at ta + i.  pre, suf: the run's values before each of its steps, and
// from the step on; start, end: where the run begins and ends.  Values of one run reach no
// other.  ACROSS: runs cross the waves (part: LDS, two entries a wave, used once), else a
// run ends with its wave.
struct Run {
    double sum;
    int cut;   // the cut that ends it (it starts from); -1: none so far
};
__device__ __forceinline__ Run joined(Run a, Run b) {   // a, then b beyond it
    return a.cut < 0 ? Run{a.sum + b.sum, b.cut} : a;
}
template <bool ACROSS>
__device__ __forceinline__ void run_sums(const double (&x)[4], unsigned cuts, int ta, int lo, int hi, Run* part,
                                         double (&pre)[4], double (&suf)[4], int (&start)[4], int (&end)[4]) {
    const int l = lane_id(), w = wave_id();
    const Run none{0.0, -1};
    auto back = [&](Run at) {   // from the steps behind the thread's to its first
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            suf[i] = x[i] + at.sum;
            end[i] = at.cut < 0 ? hi : at.cut;
            at = cuts >> i & 1 ? Run{0.0, ta + i} : Run{suf[i], at.cut};
        }
        return at;
    };
    auto ahead = [&](Run at) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (cuts >> i & 1) at = Run{0.0, ta + i};
            pre[i] = at.sum;
            start[i] = at.cut < 0 ? lo : at.cut;
            at.sum += x[i];
        }
        return at;
    };
    Run b = back(none), f = ahead(none);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const Run y{__shfl_down(b.sum, d), __shfl_down(b.cut, d)}, z{__shfl_up(f.sum, d), __shfl_up(f.cut, d)};
        if (l + d < 64) b = joined(b, y);
        if (l >= d) f = joined(f, z);
    }
    Run rb = none, rf = none;   // of the waves behind and before this one
    if constexpr (ACROSS) {
        if (l == 0) part[2 * w] = b;
        if (l == 63) part[2 * w + 1] = f;
        __syncthreads();
#pragma unroll
        for (int u = 3; u >= 0; --u)
            if (u > w) rb = joined(part[2 * u], rb);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u < w) rf = joined(part[2 * u + 1], rf);
    }
    const Run nb{__shfl_down(b.sum, 1), __shfl_down(b.cut, 1)}, nf{__shfl_up(f.sum, 1), __shfl_up(f.cut, 1)};
    back(l == 63 ? rb : joined(nb, rb));
    ahead(l == 0 ? rf : joined(nf, rf));
}

// Gate gradient of the steps t0 .. t1 - 1 that one kept state covers:
//     dg_t = B1 + sum_{t <= s < t1} (a_s - b_s),   B(t) = dg_t = e^{g_t} <S_{t - 1}, D_t>
// (the pairs that straddle t), a_s = q_s . dq_s and b_s = v_s . dv_s (= k_s . dk_s),
// summed over the channel blocks that wrote them, the pair of a step with itself left
// out.  The rounding of the differences would add up over the sequence (gradients of
// 4096 steps were off by 1e-5 of their norm).  Three things hold it down: both ends of
// a stretch are known from the kept states, and what the sum misses at t0 is taken off
// evenly along it; the pairs inside a chunk sum to zero over it, and what they sum to
// is taken off evenly along the chunk.  Sums in 64 bits.  A thread owns four steps.
// A step whose factor is below fp32's normal numbers (a reset) lets no pair through: its
// dg is zero, and the sums, their ends and what is taken off stop on either side of it, so
// that what is rounded in one document reaches no other's gradient.  NaN or Inf in a step
// of q, do or k, v reaches what lies before or behind it only: where a run's whole sum is not
// finite, each step takes the sum to whichever end is.
constexpr float kLinReset = -87.33655f;   // ln 2^-126

__device__ __forceinline__ double block_sum(double x, double* part) {   // part: one slot a wave, used once
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    if (lane_id() == 0) part[wave_id()] = x;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}
__global__ __launch_bounds__(256) void lin_dgate_kernel(LinArgs a, const float* h0, const float* s_snap,
                                                        const float* d_snap, const float* dhT, const float* dots1,
                                                        int n1, const float* dots2, int n2, float* dg) {
    __shared__ double part[2][4];
    __shared__ Run runs[8];
    const int bh = blockIdx.x / a.nent, e = blockIdx.x % a.nent, tid = threadIdx.x;
    const int n = lin_len(a.lens, bh / a.H, a.T);
    const int len = a.snap * kLinC, t0 = e * len, t1 = min(t0 + len, n);
    const int tend = min(t0 + len, a.T);
    const long row = (long)bh * a.T, se = (long)a.kd * a.nd;
    if (t0 >= n) {
        for (int t = t0 + tid; t < tend; t += 256) dg[row + t] = 0.f;
        return;
    }
    // B at step t from the state before it and the cotangent from it on (NULL: zero)
    auto straddle = [&](const float* S, const float* D, int t, double* part) {
        const float gate = t < n ? a.g[row + t] : 0.f;
        if (!S || !D || gate < kLinReset) return 0.0;
        double x = 0.0;
        constexpr int AHEAD = 8;   // pieces in flight (a state: 16 at most)
        for (int i0 = 4 * tid; i0 < (int)se; i0 += 1024 * AHEAD) {
            f32x4 u[AHEAD], v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int at = i0 + 1024 * i < (int)se ? i0 + 1024 * i : i0;
                u[i] = *reinterpret_cast<const f32x4*>(S + at);
                v[i] = *reinterpret_cast<const f32x4*>(D + at);
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (i0 + 1024 * i < (int)se)
                    x += (double)u[i][0] * v[i][0] + (double)u[i][1] * v[i][1] + (double)u[i][2] * v[i][2] +
                         (double)u[i][3] * v[i][3];
        }
        return block_sum(x, part) * (double)expf(gate);
    };
    const float* sk = s_snap + (long)bh * (a.nent + 1) * se;
    const float* dk = d_snap + (long)bh * (a.nent + 1) * se;
    const bool last = t1 >= n;   // then the cotangent is dhT and the state the last one
    const double B1 = straddle(sk + (last ? a.nent : e + 1) * se, last ? (dhT ? dhT + bh * se : nullptr) : dk + e * se,
                               last ? n : t1, part[0]);
    // the first step's gate decays h0, and nothing without one
    const double B0 = straddle(e > 0 ? sk + e * se : h0 ? h0 + bh * se : nullptr, dk + (e > 0 ? e - 1 : a.nent) * se, t0,
                               part[1]);
    const long nt = (long)a.BH * a.T;
    const int ta = t0 + 4 * tid;
    double x[4], pairs[4];
    unsigned cuts = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = pairs[i] = 0.0;
        if (ta + i >= t1) continue;
        if (ta + i > t0 && a.g[row + ta + i] < kLinReset) cuts |= 1u << i;
        for (int b = 0; b < n1; ++b) {
            const float* d = dots1 + b * nt + row + ta + i;
            x[i] += d[0];
            pairs[i] += (double)d[n1 * nt] - d[0];
        }
        for (int b = 0; b < n2; ++b) {
            const float* d = dots2 + b * nt + row + ta + i;
            x[i] -= d[0];
            pairs[i] -= (double)d[n2 * nt] - d[0];
        }
    }
    double pre[4], suf[4];
    int start[4], end[4];
    const int wt = t0 + 256 * wave_id();   // steps of this wave: whole chunks
    run_sums<false>(pairs, cuts | (ta < t1 && ta % kLinC == 0 ? 1u : 0u), ta, wt, min(wt + 256, t1), nullptr, pre, suf, start, end);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (ta + i < t1) x[i] += pairs[i] - (pre[i] + suf[i]) / (end[i] - start[i]);
    run_sums<true>(x, cuts, ta, t0, t1, runs, pre, suf, start, end);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = ta + i;
        if (t >= t1) continue;
        const double L = start[i] > t0 ? 0.0 : B0, R = end[i] < t1 ? 0.0 : B1;   // its run's ends
        const double slope = (L - (R + pre[i] + suf[i])) / (end[i] - start[i]);
        double x = R + suf[i];
        if (isfinite(slope))
            x += slope * (end[i] - t);
        else if (!isfinite(x))   // NaN or Inf in some step of the run: in one of its ends' sums only, on this side of it
            x = L - pre[i];
        dg[row + t] = t == start[i] ? (float)L : (float)x;
    }
    for (int t = t1 + tid; t < tend; t += 256) dg[row + t] = 0.f;
}

// Recurrent form: T steps of S_t = e^{g_t} S_{t-1} + v_t k_t^T, o_t = S_t q_t for every
// (b, h), the fp32 state in place.  A workgroup takes 16 state rows, 16 lanes a row
// (consecutive keys a lane), so that the state, which is nearly all the bytes of a
// single token, is read and written once in whole cache lines; S q is a DPP sum.
constexpr int kRecThreads = 256, kRecRows = 16;

template <typename T, int DK>
__global__ __launch_bounds__(kRecThreads) void lin_recurrent_kernel(const T* q, const T* k, const T* v, const float* g,
                                                                    int gate, int H, int steps, int DV, float* state,
                                                                    T* o) {
    constexpr int E = DK / 16;
    const int nblk = DV / kRecRows, bh = blockIdx.x / nblk, blk = blockIdx.x % nblk;
    const int lane = lane_id(), j = lane & 15, row = blk * kRecRows + wave_id() * 4 + (lane >> 4), c0 = j * E;
    float* srow = state + ((long)bh * DV + row) * DK + c0;
    const long tok0 = (long)bh * steps;
    float s[E], kc[E], qc[E], vc, gc;
    auto fetch = [&](int t, float(&kk)[E], float(&qq)[E], float& vv, float& gg) {
        const long tok = tok0 + t;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            kk[e] = to_f(k[tok * DK + c0 + e]);
            qq[e] = to_f(q[tok * DK + c0 + e]);
        }
        vv = to_f(v[tok * DV + row]);
        gg = gate == kLinNone ? 0.f : gate == kLinHead ? g[bh % H] : g[tok];
    };
    fetch(0, kc, qc, vc, gc);
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = srow[e];
    for (int t = 0; t < steps; ++t) {
        float kn[E], qn[E], vn, gn;
        fetch(min(t + 1, steps - 1), kn, qn, vn, gn);
        const float d = expf(gc);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s[e] = s[e] * d + vc * kc[e];
            sum += s[e] * qc[e];
        }
        sum = row16_sum(sum);
        if (j == 0) o[(tok0 + t) * DV + row] = from_f<T>(sum);
#pragma unroll
        for (int e = 0; e < E; ++e) kc[e] = kn[e], qc[e] = qn[e];
        vc = vn, gc = gn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) srow[e] = s[e];
}

template <typename T>
hipError_t rec_launch(const LinProblem& pr, const void* q, const void* k, const void* v, const float* g, float* state,
                      void* o, hipStream_t s) {
    const dim3 grid((unsigned)((long)pr.B * pr.H * (pr.dv / kRecRows))), block(kRecThreads);
#define DN_REC(D)                                                                                                   \
    case D:                                                                                                         \
        hipLaunchKernelGGL((lin_recurrent_kernel<T, D>), grid, block, 0, s, static_cast<const T*>(q),               \
                           static_cast<const T*>(k), static_cast<const T*>(v), g, pr.gate, pr.H, pr.T, pr.dv, state, \
                           static_cast<T*>(o));                                                                     \
        break;
    switch (pr.dk) {
        DN_REC(16)
        DN_REC(32)
        DN_REC(64)
        DN_REC(128)
        default: return hipErrorInvalidValue;
    }
#undef DN_REC
    return hipGetLastError();
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }
int ceil_div(int a, int b) { return (a + b - 1) / b; }
int blocks_of(int nd, int bf16) { return nd / lin_vb(nd, bf16 != 0); }

// Time of a launch of segments of len chunks, in chunks of one workgroup alone on its unit:
// `per` workgroups for each (b, h) and segment, whose units (bh, segment) go to the 8 XCDs in
// turn, so that the fullest XCD counts; two workgroups on a unit take 1.7 of one's time, and each
// begins with a chunk's worth of loads.  The pass that makes the segments' own states (`state`
// workgroups in all) takes half as much for a chunk and fits a unit more often.
float segments_time(long units, int per, int len, long state) {
    const long k = ((units + kXcds - 1) / kXcds * per + kLinUnits / kXcds - 1) / (kLinUnits / kXcds);
    const float outs = 1.7f * (float)(k / 2) + (float)(k % 2), states = std::max(1.f, (float)state / (2 * kLinUnits));
    return (len + 1) * (outs + 0.5f * states);
}

// Parallel segments of the steps.  One run of all chunks reads every tensor once and takes
// a time that grows with the chunks alone while a compute unit has at most one workgroup;
// segments fill the units, at the cost of a pass over the two tensors of the state, the
// boundary states and two launches.  With w workgroups in one run, segments take
// w / full of its time per chunk and `cost` chunks more.  Measured (one run -> the best of 2 to 64
// segments, d = 128):
//     bf16 outputs, NT 256      w  96 503 -> 339 us, 128: 500 -> 453; 192 (NT 512): 1012 -> 1154
//     bf16, gate's gradient, NT 256  w  96 1360 -> 630 us, 200: 1442 -> 1303
//     fp32 outputs, NT 256      w  96 1223 -> 615 us, 128: 1230 -> 804; gate's gradient, w 240: 3045 -> 2785
// Where the fullest XCD has workgroups for two turns of its units although all together would
// fit in one (fp32, 20 heads x 12 workgroups: 2430 us in one run, 1454 in 5 segments), w counts
// half.  The number of segments is then the fastest by segments_time, of the lengths that there
// are after rounding (with the gate's gradient to whole numbers of kept states): over 2 to 64
// segments of 6 to 240 workgroups, 16 to 256 chunks, d = 32, 64 and 128, within 2 % of the best
// on average (filling four workgroups a unit: 3.5 %).  Segments are of at least 4 chunks, or,
// while those leave units idle, of 2.
LinPlan lin_plan(const LinProblem& pr, int nops, bool dots) {
    const int NT = ceil_div(pr.T, kLinC), nblk = blocks_of(pr.dv, pr.bf16);
    const long BH = (long)pr.B * pr.H, wgs = BH * nblk * nops;
    const long full = pr.bf16 ? (dots ? 216 : 144) : (dots ? 256 : 208), cost = pr.bf16 ? (dots ? 6 : 9) : 4;
    const long fullest = (BH + kXcds - 1) / kXcds * kXcds * nblk * nops;
    const long w = wgs <= kLinUnits && fullest > kLinUnits ? wgs / 2 : wgs;
    // kept states of a segment of len chunks: at equal distances, at most kLinSnap
    auto distance = [&](int len) { return ceil_div(len, ceil_div(len, kLinSnap)); };
    LinPlan p;
    p.nseg = 1;
    p.seg_len = std::max(NT, 1);
    p.snap = dots ? kLinSnap : p.seg_len;
    if (!pr.no_scan && wgs > 0 && NT * (full - w) >= cost * full) {
        const int most = (int)std::min<long>({kLinMaxSeg, NT / 2, 8 * kLinUnits / wgs});
        float best = 0.f;
        for (int ns = 2; ns <= most; ++ns) {
            int len = ceil_div(NT, ns);
            const int snap = dots ? distance(len) : len;
            len = ceil_div(len, snap) * snap;
            const int nseg = ceil_div(NT, len);
            if (nseg < 2 || (len < 4 && nseg * wgs > kLinUnits)) continue;
            const float time = segments_time(BH * nseg, nblk * nops, len, BH * (nseg - 1) * nblk * (nops > 1 ? 2 : 1));
            if (p.nseg > 1 && time >= best) continue;
            best = time;
            p.nseg = nseg, p.seg_len = len, p.snap = snap;
        }
    }
    p.nent = NT > 0 ? ceil_div(NT, p.snap) : 1;
    return p;
}

// Evaluations that share a launch in the backward.
int bwd_ops(bool dots) { return dots ? 2 : 3; }

const LinLaunch kLaunch[2][3] = {{lin_f32_k32, lin_f32_k64, lin_f32_k128}, {lin_bf16_k32, lin_bf16_k64, lin_bf16_k128}};

hipError_t launch_chunks(const LinProblem& pr, const LinArgs& a, int mode, hipStream_t s) {
    const int ki = a.kd <= 32 ? 0 : a.kd == 64 ? 1 : 2;
    return kLaunch[pr.bf16 ? 1 : 0][ki](a, lin_vb(a.nd, pr.bf16 != 0) / 16, mode, s);
}

LinArgs base_args(const LinProblem& pr, const LinPlan& pl, const float* g, const int* lens) {
    LinArgs a{};
    a.BH = pr.B * pr.H;
    a.H = pr.H;
    a.T = pr.T;
    a.NT = ceil_div(pr.T, kLinC);
    a.nseg = pl.nseg;
    a.seg_len = pl.seg_len;
    a.snap = pl.snap;
    a.nent = pl.nent;
    a.g = g;
    a.gate = pr.gate;
    a.lens = lens;
    return a;
}

void set_dims(LinArgs& a, const LinProblem& pr, int kd, int nd) {
    a.kd = kd;
    a.nd = nd;
    a.nblk = blocks_of(nd, pr.bf16);
}

// Boundary states of every op of `a` (their y, z, init, snap, rev).
hipError_t launch_boundaries(const LinProblem& pr, LinArgs a, hipStream_t s) {
    prof_begin(s, "linear_segments");
    hipError_t e = launch_chunks(pr, a, kLinState, s);
    prof_end(s);
    if (e != hipSuccess) return e;
    prof_begin(s, "linear_join");
    const dim3 grid((unsigned)(a.BH * (a.kd * a.nd / 256)), a.nops), block(256);
    if (a.nseg <= 8)
        hipLaunchKernelGGL(lin_join_kernel<8>, grid, block, 0, s, a);
    else if (a.nseg <= 16)
        hipLaunchKernelGGL(lin_join_kernel<16>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(lin_join_kernel<kLinMaxSeg>, grid, block, 0, s, a);
    prof_end(s);
    return hipGetLastError();
}

struct LinWs {
    size_t s_snap, d_snap, segdec, dots1, dots2, total;
};
LinWs lin_ws(const LinProblem& pr, int pass) {
    const size_t BH = (size_t)pr.B * pr.H, se = (size_t)pr.dk * pr.dv * 4;
    const bool bwd = pass != 0, dots = bwd && pr.gate == kLinScalar;
    const LinPlan p = lin_plan(pr, bwd ? bwd_ops(dots) : 1, dots);
    const bool keep = p.nseg > 1 || dots;
    LinWs w{};
    size_t off = 0;
    w.s_snap = off;
    off += keep ? al256(BH * (p.nent + 1) * se) : 0;
    w.d_snap = off;
    off += keep && bwd ? al256(BH * (p.nent + 1) * se) : 0;
    w.segdec = off;
    off += p.nseg > 1 ? al256((bwd ? 2 : 1) * BH * p.nseg * 4) : 0;
    w.dots1 = off;
    off += dots ? al256(2 * (size_t)blocks_of(pr.dk, pr.bf16) * BH * pr.T * 4) : 0;
    w.dots2 = off;
    off += dots ? al256(2 * (size_t)blocks_of(pr.dv, pr.bf16) * BH * pr.T * 4) : 0;
    w.total = off;
    return w;
}

}  // namespace

size_t lin_workspace_bytes(const LinProblem& pr, int pass) { return lin_ws(pr, pass).total; }

hipError_t launch_linear_fwd(const LinProblem& pr, const LinFwd& f, char* ws, hipStream_t s) {
    if (pr.B * pr.H == 0) return hipSuccess;
    const LinPlan pl = lin_plan(pr, 1, false);
    const LinWs w = lin_ws(pr, 0);
    LinArgs a = base_args(pr, pl, f.g, f.lens);
    set_dims(a, pr, pr.dk, pr.dv);
    LinOp& op = a.op[0];
    op.x = f.q;
    op.y = f.k;
    op.z = f.v;
    op.out = f.o;
    op.init = f.h0;
    op.fin = f.hT;
    op.snap = pl.nseg > 1 ? reinterpret_cast<float*>(ws + w.s_snap) : nullptr;
    op.snap_bh = (long)(pl.nent + 1) * pr.dk * pr.dv;
    op.sn = pr.dk;
    op.sk = 1;
    a.nops = 1;
    a.segdec = reinterpret_cast<float*>(ws + w.segdec);
    if (pl.nseg > 1) {
        const hipError_t e = launch_boundaries(pr, a, s);
        if (e != hipSuccess) return e;
    }
    prof_begin(s, "linear_fwd");
    const hipError_t e = launch_chunks(pr, a, kLinOut, s);
    prof_end(s);
    return e;
}

hipError_t launch_linear_bwd(const LinProblem& pr, const LinBwd& f, char* ws, hipStream_t s) {
    if (pr.B * pr.H == 0) return hipSuccess;
    const bool dots = pr.gate == kLinScalar;
    const LinPlan pl = lin_plan(pr, bwd_ops(dots), dots);
    const LinWs w = lin_ws(pr, 1);
    const bool keep = pl.nseg > 1 || dots;
    float* s_snap = keep ? reinterpret_cast<float*>(ws + w.s_snap) : nullptr;
    float* d_snap = keep ? reinterpret_cast<float*>(ws + w.d_snap) : nullptr;
    const long se = (long)pr.dk * pr.dv;
    LinArgs base = base_args(pr, pl, f.g, f.lens);
    base.segdec = reinterpret_cast<float*>(ws + w.segdec);
    LinOp dq{}, dk{}, dv{};
    dq.x = f.dout, dq.y = f.v, dq.z = f.k, dq.out = f.dq;
    dq.init = f.h0, dq.snap = s_snap, dq.snap_bh = (pl.nent + 1) * se, dq.sn = 1, dq.sk = pr.dk;
    dv.x = f.k, dv.y = f.q, dv.z = f.dout, dv.out = f.dv, dv.rev = 1;
    dv.init = f.dhT, dv.fin = f.dh0, dv.snap = d_snap, dv.snap_bh = (pl.nent + 1) * se, dv.sn = pr.dk, dv.sk = 1;
    dk.x = f.v, dk.y = f.dout, dk.z = f.q, dk.out = f.dk, dk.rev = 1;
    dk.init = f.dhT, dk.snap = d_snap, dk.snap_bh = (pl.nent + 1) * se, dk.sn = 1, dk.sk = pr.dk;
    hipError_t e = hipSuccess;
    if (pl.nseg > 1) {
        LinArgs a = base;
        set_dims(a, pr, pr.dk, pr.dv);
        a.nops = 2;
        a.op[0] = dv;
        a.op[1] = dv;
        a.op[0].y = f.k, a.op[0].z = f.v, a.op[0].init = f.h0, a.op[0].rev = 0;
        a.op[0].snap = s_snap, a.op[0].snap_bh = dq.snap_bh;
        if ((e = launch_boundaries(pr, a, s)) != hipSuccess) return e;
    }
    if (dots) {
        dq.r = f.q, dq.dots = reinterpret_cast<float*>(ws + w.dots1);
        dv.r = f.v, dv.dots = reinterpret_cast<float*>(ws + w.dots2);
    }
    // evaluations of the same widths and mode share a launch (and their rows in L2)
    auto run = [&](const LinOp* ops, int n, int kd, int nd, int mode) {
        LinArgs a = base;
        set_dims(a, pr, kd, nd);
        a.nops = n;
        for (int i = 0; i < n; ++i) a.op[i] = ops[i];
        return launch_chunks(pr, a, mode, s);
    };
    const int mode = dots ? kLinDots : kLinOut;
    prof_begin(s, "linear_bwd");
    if (pr.dk == pr.dv && !dots) {
        const LinOp all[3] = {dq, dk, dv};
        e = run(all, 3, pr.dk, pr.dv, mode);
    } else if (pr.dk == pr.dv) {
        const LinOp two[2] = {dq, dv};
        e = run(two, 2, pr.dk, pr.dv, mode);
        if (e == hipSuccess) e = run(&dk, 1, pr.dv, pr.dk, kLinOut);
    } else {
        if (dots) {
            e = run(&dq, 1, pr.dv, pr.dk, mode);
            if (e == hipSuccess) e = run(&dk, 1, pr.dv, pr.dk, kLinOut);
        } else {
            const LinOp two[2] = {dq, dk};
            e = run(two, 2, pr.dv, pr.dk, mode);
        }
        if (e == hipSuccess) e = run(&dv, 1, pr.dk, pr.dv, mode);
    }
    prof_end(s);
    if (e != hipSuccess || !dots || pr.T == 0) return e;
    prof_begin(s, "linear_dgate");
    set_dims(base, pr, pr.dk, pr.dv);
    hipLaunchKernelGGL(lin_dgate_kernel, dim3((unsigned)(base.BH * pl.nent)), dim3(256), 0, s, base, f.h0, s_snap, d_snap,
                       f.dhT, dq.dots, blocks_of(pr.dk, pr.bf16), dv.dots, blocks_of(pr.dv, pr.bf16), f.dg);
    prof_end(s);
    return hipGetLastError();
}

hipError_t launch_linear_recurrent(const LinProblem& pr, const void* q, const void* k, const void* v, const float* g,
                                   float* state, void* o, hipStream_t s) {
    if ((long)pr.B * pr.H * pr.T == 0) return hipSuccess;
    prof_begin(s, "linear_recurrent");
    const hipError_t e = pr.bf16 ? rec_launch<bf16>(pr, q, k, v, g, state, o, s)
                                 : rec_launch<float>(pr, q, k, v, g, state, o, s);
    prof_end(s);
    return e;
}

}  // namespace dn
