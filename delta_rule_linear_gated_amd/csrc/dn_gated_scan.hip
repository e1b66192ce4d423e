// dn_gated_scan.hip -- gated linear recurrence, one state a channel:
//     h_t = e^{g_t} h_{t-1} + w_t x_t,   o_t = h_t,   w_t = 1 or (coupled) 1 - e^{g_t},
// its backward pass and its recurrent form.  Layouts as in include/dn.h.
//
// A step is the affine map h -> a h + b; a run of steps is the map {p, e}, p the product of
// its decays and e its end from a zero state.  A workgroup owns a strip of 64 channels (a
// lane each) and walks the steps in tiles: each of its 16 waves forms the map of its run of
// the tile in registers, the waves exchange the maps through LDS (one barrier a tile), each
// takes its run's first state through the maps before it and goes over its registers again
// for the outputs.  All of a tile's rows are loaded while the one before is worked on, so
// that every tensor is read once.  Strips alone fill the chip from 256 on; fewer are cut
// into segments of the steps, whose maps a pass of its own forms first (gs_plan).
//
// The backward walks the same tiles from the last step with r_t = a_t D_t, the cotangent
// that leaves step t to earlier ones:
//     D_t = do_t + r_{t+1},   dx_t = w_t D_t,   dg_t = r_t (h_{t-1} - [coupled] x_t),
// h inside a tile from the state saved at its start.
#include <algorithm>

#include "dn_device.h"
#include "dn_gated_scan.h"
#include "dn_internal.h"

namespace dn {

namespace {

constexpr int kGsWaves = 16;
constexpr int kGsRun = 16;                        // steps of a wave in a tile, forward
constexpr int kGsRunB = kGsSaved / kGsWaves;      // and backward: a tile begins at a saved state
constexpr int kGsTile = kGsWaves * kGsRun;
constexpr int kGsMaxSeg = 64;
constexpr int kGsUnits = 256;                     // compute units
static_assert(kGsTile % kGsSaved == 0, "saved states lie at the starts of runs");
constexpr int kRange = 0x7fffff00;                // bytes of a buffer range, at most
constexpr int kNowhere = 0x7ffffff0;              // an offset past every range: loads give zero, stores do nothing

struct GsArgs {
    int BH, H, T, d;
    int strips, nseg, seg_len;   // seg_len: steps
    int flat;                    // channel of a lane: 64 strip + lane of all, else of one head's row
    int NS;                      // saved states of a row
    const void *x, *y;           // y: dout
    const float* g;
    const int* lens;
    const float *first, *states_in;
    float2* maps;                // [nseg][strips][64] of the segments
    void* out;                   // o or dx; NULL: not wanted
    float *dg, *last, *states;
};

// The channel of a lane, and where its row begins in the strip.
struct Lane {
    long row;      // (b, h)
    int c, off;    // channel; elements from the strip's first row to the lane's channel
    int len;       // steps of its sequence, 0 for an idle lane
    bool on;
};
__device__ __forceinline__ Lane gs_lane(const GsArgs& a, int strip, long& row0) {
    Lane l;
    const int lane = lane_id();
    if (a.flat) {
        const long n0 = 64L * strip, n = n0 + lane;
        row0 = n0 / a.d;
        l.row = n / a.d;
        l.c = (int)(n - l.row * a.d);
        l.on = l.row < a.BH;
    } else {
        const int per = (a.d + 63) / 64;
        row0 = l.row = strip / per;
        l.c = strip % per * 64 + lane;
        l.on = l.c < a.d;
    }
    l.off = l.on ? (int)(l.row - row0) * a.T * a.d + l.c : 0;
    l.len = !l.on ? 0 : a.lens ? min(max(a.lens[l.row / a.H], 0), a.T) : a.T;
    return l;
}

// What lies from element `at` on of a tensor of n elements, as a buffer.
template <typename T> __device__ __forceinline__ __amdgpu_buffer_rsrc_t gs_range(const void* p, long n, long at) {
    const long left = (n - at) * (long)sizeof(T);
    const int bytes = left <= 0 ? 0 : left < kRange ? (int)left : kRange;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(static_cast<const T*>(p) + (left > 0 ? at : 0)), (short)0,
                                             bytes, 0x00020000);
}
template <typename T> struct Bits;
template <> struct Bits<float> {
    static __device__ __forceinline__ unsigned load(__amdgpu_buffer_rsrc_t r, int at, int s) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, at, s, 0);
    }
    static __device__ __forceinline__ float value(unsigned u) { return __builtin_bit_cast(float, u); }
    static __device__ __forceinline__ void store(float v, __amdgpu_buffer_rsrc_t r, int at, int s) {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, at, s, 0);
    }
};
template <> struct Bits<bf16> {
    static __device__ __forceinline__ unsigned load(__amdgpu_buffer_rsrc_t r, int at, int s) {
        return __builtin_amdgcn_raw_buffer_load_b16(r, at, s, 0);
    }
    static __device__ __forceinline__ float value(unsigned u) { return __builtin_bit_cast(float, u << 16); }
    static __device__ __forceinline__ void store(float v, __amdgpu_buffer_rsrc_t r, int at, int s) {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, from_f<bf16>(v)), r, at, s, 0);
    }
};

// R rows of a strip from step t on, a step's value in a register.  Rows past a lane's `end`
// read as zero (g: a factor of one) and are not written.  All of a wave's lanes full (the
// wave asks with __all): the steps are scalar offsets, else selects.
template <typename T, int R>
__device__ __forceinline__ void gs_load(unsigned (&v)[R], const void* p, const GsArgs& a, long row0, const Lane& l,
                                        int t, int end, bool full) {
    const long n = (long)a.BH * a.T * a.d, at = (row0 * a.T + t) * a.d;
    const auto r = gs_range<T>(p, n, at);
    const int step = a.d * (int)sizeof(T), off = l.on ? l.off * (int)sizeof(T) : kNowhere;
    if (full) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = Bits<T>::load(r, off, i * step);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = Bits<T>::load(r, t + i < end ? off + i * step : kNowhere, 0);
    }
}
// A lane's rows from its `end` up to T are written as zero.
template <typename T, int R>
__device__ __forceinline__ void gs_store(const float (&v)[R], void* p, const GsArgs& a, long row0, const Lane& l, int t,
                                         int end, bool full) {
    const long n = (long)a.BH * a.T * a.d, at = (row0 * a.T + t) * a.d;
    const auto r = gs_range<T>(p, n, at);
    const int step = a.d * (int)sizeof(T), off = l.on ? l.off * (int)sizeof(T) : kNowhere;
    if (full) {
#pragma unroll
        for (int i = 0; i < R; ++i) Bits<T>::store(v[i], r, off, i * step);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            Bits<T>::store(t + i < end ? v[i] : 0.f, r, l.on && t + i < a.T ? off + i * step : kNowhere, 0);
    }
}

constexpr float kLog2e = 1.44269504088896341f;
__device__ __forceinline__ float gs_exp(float g) { return __builtin_amdgcn_exp2f(g * kLog2e); }
// 1 - e^g with a = e^g: by its series within 1/2, where the difference would lose the bits
// that a shares with 1 (the eighth term leaves 1e-8 of the value).
__device__ __forceinline__ float gs_rest(float g, float a) {
    float s = 1.f / 40320.f;
    s = fmaf(s, g, 1.f / 5040.f);
    s = fmaf(s, g, 1.f / 720.f);
    s = fmaf(s, g, 1.f / 120.f);
    s = fmaf(s, g, 1.f / 24.f);
    s = fmaf(s, g, 1.f / 6.f);
    s = fmaf(s, g, 0.5f);
    s = fmaf(s, g, 1.f);
    return fabsf(g) < 0.5f ? -g * s : 1.f - a;
}

__device__ __forceinline__ int uniform_wave() { return __builtin_amdgcn_readfirstlane(wave_id()); }

// The state that enters the strip's segment, through the maps of the segments before it
// (REV: behind it), shared by the waves.
template <bool REV> __device__ __forceinline__ float gs_enter(const GsArgs& a, int strip, int seg, float first,
                                                              float2 (*part)[64]) {
    const int w = uniform_wave(), l = lane_id();
    const int before = REV ? a.nseg - 1 - seg : seg;
    if (before == 0) return first;
    const int per = (before + kGsWaves - 1) / kGsWaves;
    float2 m[kGsMaxSeg / kGsWaves];
#pragma unroll
    for (int i = 0; i < kGsMaxSeg / kGsWaves; ++i) {
        const int s = min(w * per + i, before - 1);
        m[i] = a.maps[((long)(REV ? a.nseg - 1 - s : s) * a.strips + strip) * 64 + l];
    }
    float p = 1.f, e = 0.f;
#pragma unroll
    for (int i = 0; i < kGsMaxSeg / kGsWaves; ++i)
        if (i < per && w * per + i < before) {
            p *= m[i].x;
            e = fmaf(m[i].x, e, m[i].y);
        }
    part[w][l] = make_float2(p, e);
    __syncthreads();
    float h = first;
#pragma unroll
    for (int v = 0; v < kGsWaves; ++v) h = fmaf(part[v][l].x, h, part[v][l].y);
    __syncthreads();
    return h;
}

// Forward.  MAPS: the segment's map only (all but the last segment); else outputs, saved
// states and the last state, each where wanted.
template <typename T, bool COUPLED, bool MAPS>
__global__ __launch_bounds__(64 * kGsWaves) void gated_scan_fwd_kernel(GsArgs a) {
    __shared__ float2 part[2][kGsWaves][64];
    const int strip = blockIdx.x % a.strips, seg = blockIdx.x / a.strips;
    const int w = uniform_wave(), lane = lane_id();
    long row0;
    const Lane l = gs_lane(a, strip, row0);
    const int begin = seg * a.seg_len, end = min(a.T, begin + a.seg_len), len = min(l.len, end);
    constexpr int R = kGsRun;
    float h = !MAPS && a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f, p = 1.f;
    if (!MAPS) h = gs_enter<false>(a, strip, seg, h, part[0]);
    unsigned gn[R], xn[R];
    auto fetch = [&](int t) {
        const bool full = __all(!l.on || len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, len, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, len, full);
    };
    int t0 = begin, buf = 0;
    if (__any(len > t0)) fetch(t0 + w * R);
    for (; __any(len > t0); t0 += kGsTile, buf ^= 1) {
        const int t = t0 + w * R;
        float f[R], b[R], sum = 0.f, e = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float g = Bits<float>::value(gn[i]);
            b[i] = Bits<T>::value(xn[i]);
            f[i] = gs_exp(g);
            if (COUPLED) b[i] *= gs_rest(g, f[i]);
            sum += g;
            e = fmaf(f[i], e, b[i]);
        }
        if (__any(len > t0 + kGsTile)) fetch(t + kGsTile);
        part[buf][w][lane] = make_float2(gs_exp(sum), e);
        __syncthreads();
        float mine = h;
#pragma unroll
        for (int v = 0; v < kGsWaves; ++v) {
            const float2 m = part[buf][v][lane];
            if (v == w) mine = h;
            h = fmaf(m.x, h, m.y);
            if (MAPS) p *= m.x;
        }
        if (MAPS) continue;
        if (a.states && l.on && t % kGsSaved == 0 && t < end) a.states[(l.row * a.NS + t / kGsSaved) * a.d + l.c] = mine;
        if (!a.out) continue;
        const bool full = __all(!l.on || len >= t + R);
#pragma unroll
        for (int i = 0; i < R; ++i) b[i] = mine = fmaf(f[i], mine, b[i]);
        gs_store<T, R>(b, a.out, a, row0, l, t, len, full);
    }
    if (MAPS) {
        if (w == 0) a.maps[((long)seg * a.strips + strip) * 64 + lane] = make_float2(p, h);
        return;
    }
    if (a.out) {   // the tiles that no sequence of the strip reaches
        float none[R] = {};
        for (; t0 < end; t0 += kGsTile) gs_store<T, R>(none, a.out, a, row0, l, t0 + w * R, len, false);
    }
    if (a.last && seg == a.nseg - 1 && w == 0 && l.on) a.last[l.row * a.d + l.c] = h;
}

// The maps of the segments from their last step back: r -> a (r + do).
template <typename T> __global__ __launch_bounds__(64 * kGsWaves) void gated_scan_back_kernel(GsArgs a) {
    __shared__ float2 part[2][kGsWaves][64];
    const int strip = blockIdx.x % a.strips, seg = blockIdx.x / a.strips + 1;
    const int w = uniform_wave(), lane = lane_id();
    long row0;
    const Lane l = gs_lane(a, strip, row0);
    const int begin = seg * a.seg_len, end = min(a.T, begin + a.seg_len), len = min(l.len, end);
    constexpr int R = kGsRun;
    float r = 0.f, p = 1.f;
    unsigned gn[R], yn[R];
    auto fetch = [&](int t) {
        const bool full = __all(!l.on || len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, len, full);
        gs_load<T, R>(yn, a.y, a, row0, l, t, len, full);
    };
    int t0 = begin + (end - begin - 1) / kGsTile * kGsTile, buf = 0;
    while (t0 >= begin && !__any(len > t0)) t0 -= kGsTile;
    if (t0 >= begin) fetch(t0 + w * R);
    for (; t0 >= begin; t0 -= kGsTile, buf ^= 1) {
        float f[R], y[R], sum = 0.f, e = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float g = Bits<float>::value(gn[i]);
            f[i] = gs_exp(g);
            y[i] = Bits<T>::value(yn[i]);
            sum += g;
        }
        if (t0 > begin) fetch(t0 - kGsTile + w * R);
#pragma unroll
        for (int i = R - 1; i >= 0; --i) e = f[i] * (e + y[i]);
        part[buf][w][lane] = make_float2(gs_exp(sum), e);
        __syncthreads();
#pragma unroll
        for (int v = kGsWaves - 1; v >= 0; --v) {
            const float2 m = part[buf][v][lane];
            r = fmaf(m.x, r, m.y);
            p *= m.x;
        }
    }
    if (w == 0) a.maps[((long)seg * a.strips + strip) * 64 + lane] = make_float2(p, r);
}

template <typename T, bool COUPLED>
__global__ __launch_bounds__(64 * kGsWaves) void gated_scan_bwd_kernel(GsArgs a) {
    __shared__ float2 ahead[2][kGsWaves][64], back[2][kGsWaves][64];
    const int strip = blockIdx.x % a.strips, seg = blockIdx.x / a.strips;
    const int w = uniform_wave(), lane = lane_id();
    long row0;
    const Lane l = gs_lane(a, strip, row0);
    const int begin = seg * a.seg_len, end = min(a.T, begin + a.seg_len), len = min(l.len, end);
    constexpr int R = kGsRunB;
    constexpr int TILE = kGsWaves * R;
    float r = a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f;
    r = gs_enter<true>(a, strip, seg, r, back[0]);
    unsigned gn[R], xn[R], yn[R];
    float hn;
    auto fetch = [&](int t0) {
        const int t = t0 + w * R;
        const bool full = __all(!l.on || len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, len, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, len, full);
        gs_load<T, R>(yn, a.y, a, row0, l, t, len, full);
        hn = len > t0 ? a.states_in[(l.row * a.NS + t0 / kGsSaved) * a.d + l.c] : 0.f;
    };
    int t0 = begin + (end > begin ? (end - begin - 1) / TILE * TILE : -TILE), buf = 0;
    for (float none[R] = {}; t0 >= begin && !__any(len > t0); t0 -= TILE) {
        gs_store<T, R>(none, a.out, a, row0, l, t0 + w * R, len, false);
        gs_store<float, R>(none, a.dg, a, row0, l, t0 + w * R, len, false);
    }
    if (t0 >= begin) fetch(t0);
    for (; t0 >= begin; t0 -= TILE, buf ^= 1) {
        const int t = t0 + w * R;
        float f[R], x[R], y[R], wt[R], h = hn, sum = 0.f, e = 0.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float g = Bits<float>::value(gn[i]);
            x[i] = Bits<T>::value(xn[i]);
            y[i] = Bits<T>::value(yn[i]);
            f[i] = gs_exp(g);
            wt[i] = COUPLED ? gs_rest(g, f[i]) : 1.f;
            sum += g;
            e = fmaf(f[i], e, wt[i] * x[i]);
        }
        if (t0 > begin) fetch(t0 - TILE);
#pragma unroll
        for (int i = R - 1; i >= 0; --i) q = f[i] * (q + y[i]);
        const float p = gs_exp(sum);
        ahead[buf][w][lane] = make_float2(p, e);
        back[buf][w][lane] = make_float2(p, q);
        __syncthreads();
        float mine = r;
#pragma unroll
        for (int v = kGsWaves - 1; v >= 0; --v) {
            const float2 m = back[buf][v][lane];
            if (v == w) mine = r;
            r = fmaf(m.x, r, m.y);
        }
#pragma unroll
        for (int v = 0; v < kGsWaves - 1; ++v)
            if (v < w) {
                const float2 m = ahead[buf][v][lane];
                h = fmaf(m.x, h, m.y);
            }
        float before[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            before[i] = COUPLED ? h - x[i] : h;
            h = fmaf(f[i], h, wt[i] * x[i]);
        }
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            const float D = y[i] + mine;
            mine = f[i] * D;
            x[i] = COUPLED ? wt[i] * D : D;
            y[i] = mine * before[i];
        }
        const bool full = __all(!l.on || len >= t + R);
        gs_store<T, R>(x, a.out, a, row0, l, t, len, full);
        gs_store<float, R>(y, a.dg, a, row0, l, t, len, full);
    }
    if (a.last && seg == 0 && w == 0 && l.on) a.last[l.row * a.d + l.c] = r;
}

// Recurrent form: a thread a channel, the state in a register over the steps; bytes and
// latency of its few rows are all there is to it.
template <typename T, bool COUPLED>
__global__ __launch_bounds__(256) void gated_scan_recurrent_kernel(const T* x, const float* g, float* state, T* o, int BH,
                                                                   int steps, int d) {
    const long n = blockIdx.x * 256L + threadIdx.x, row = n / d;
    if (row >= BH) return;
    const long at = row * steps * d + (n - row * d);
    float h = state[n], gn = g[at], xn = to_f(x[at]);
    for (int t = 0; t < steps; ++t) {
        const float gc = gn, xc = xn;
        if (t + 1 < steps) gn = g[at + (t + 1L) * d], xn = to_f(x[at + (t + 1L) * d]);
        const float f = gs_exp(gc);
        h = fmaf(f, h, COUPLED ? gs_rest(gc, f) * xc : xc);
        o[at + (long)t * d] = from_f<T>(h);
    }
    state[n] = h;
}

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

struct GsPlan {
    int flat, nseg, seg_len;
    long strips;
};

// Lanes take the channels of all heads in a row, so that odd widths leave no lane idle but the
// last strip's; where a strip's rows lie further apart than a 31-bit byte offset, a strip stays
// in one head's row.
void gs_strips(const GsProblem& pr, GsPlan* p) {
    const long BH = (long)pr.B * pr.H, rows = 63 / pr.d + 2;   // a strip touches at most that many
    p->flat = rows * pr.T < kRange / 4 / pr.d;
    p->strips = p->flat ? (BH * pr.d + 63) / 64 : BH * ((pr.d + 63) / 64);
}
GsPlan gs_plan(const GsProblem& pr) {
    GsPlan p;
    gs_strips(pr, &p);
    const int tiles = (int)(((long)pr.T + kGsTile - 1) / kGsTile);
    int nseg = 1;
    if (p.strips > 0 && p.strips < kGsUnits && tiles >= 4)
        nseg = (int)std::min<long>({kGsMaxSeg, tiles / 2, (kGsUnits + p.strips - 1) / p.strips});
    const int len = tiles > 0 ? (tiles + nseg - 1) / nseg : 1;
    p.nseg = tiles > 0 ? (tiles + len - 1) / len : 1;
    p.seg_len = (int)std::min<long>((long)len * kGsTile, 0x7fffff00);
    return p;
}

struct GsWs {
    size_t maps, states, total;
};
GsWs gs_ws(const GsProblem& pr, int pass) {
    const GsPlan p = gs_plan(pr);
    GsWs w{};
    w.states = p.nseg > 1 ? al256((size_t)p.nseg * p.strips * 64 * 8) : 0;
    w.total = w.states + (pass == 2 ? al256(gs_states_bytes(pr)) : 0);
    return w;
}

GsArgs gs_args(const GsProblem& pr, const GsPlan& p, const void* x, const float* g, const int* lens, char* ws) {
    GsArgs a{};
    a.BH = pr.B * pr.H;
    a.H = pr.H;
    a.T = pr.T;
    a.d = pr.d;
    a.strips = (int)p.strips;
    a.nseg = p.nseg;
    a.seg_len = p.seg_len;
    a.flat = p.flat;
    a.NS = (int)(((long)pr.T + kGsSaved - 1) / kGsSaved);
    a.x = x;
    a.g = g;
    a.lens = lens;
    a.maps = reinterpret_cast<float2*>(ws);
    return a;
}

template <typename T, bool COUPLED> hipError_t fwd_launch(const GsArgs& a, hipStream_t s) {
    const dim3 block(64 * kGsWaves);
    if (a.nseg > 1) {
        prof_begin(s, "gated_scan_maps");
        hipLaunchKernelGGL((gated_scan_fwd_kernel<T, COUPLED, true>), dim3(a.strips * (a.nseg - 1)), block, 0, s, a);
        prof_end(s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    prof_begin(s, "gated_scan_fwd");
    hipLaunchKernelGGL((gated_scan_fwd_kernel<T, COUPLED, false>), dim3(a.strips * a.nseg), block, 0, s, a);
    prof_end(s);
    return hipGetLastError();
}
template <typename T, bool COUPLED> hipError_t bwd_launch(const GsArgs& a, hipStream_t s) {
    const dim3 block(64 * kGsWaves);
    if (a.nseg > 1) {
        prof_begin(s, "gated_scan_back");
        hipLaunchKernelGGL((gated_scan_back_kernel<T>), dim3(a.strips * (a.nseg - 1)), block, 0, s, a);
        prof_end(s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    prof_begin(s, "gated_scan_bwd");
    hipLaunchKernelGGL((gated_scan_bwd_kernel<T, COUPLED>), dim3(a.strips * a.nseg), block, 0, s, a);
    prof_end(s);
    return hipGetLastError();
}
hipError_t fwd_any(const GsProblem& pr, const GsArgs& a, hipStream_t s) {
    if (pr.bf16) return pr.coupled ? fwd_launch<bf16, true>(a, s) : fwd_launch<bf16, false>(a, s);
    return pr.coupled ? fwd_launch<float, true>(a, s) : fwd_launch<float, false>(a, s);
}
hipError_t bwd_any(const GsProblem& pr, const GsArgs& a, hipStream_t s) {
    if (pr.bf16) return pr.coupled ? bwd_launch<bf16, true>(a, s) : bwd_launch<bf16, false>(a, s);
    return pr.coupled ? bwd_launch<float, true>(a, s) : bwd_launch<float, false>(a, s);
}

}  // namespace

size_t gs_states_bytes(const GsProblem& pr) {
    return (size_t)pr.B * pr.H * (((size_t)pr.T + kGsSaved - 1) / kGsSaved) * pr.d * 4;
}
size_t gs_workspace_bytes(const GsProblem& pr, int pass) { return gs_ws(pr, pass).total; }
bool gs_fits(const GsProblem& pr) {
    if (pr.B == 0 || pr.H == 0) return true;
    GsPlan p;
    gs_strips(pr, &p);
    return (long)pr.B * pr.H <= 0x7fffffffL && p.strips < (1L << 32) / (64 * kGsWaves);
}

hipError_t launch_gated_scan_fwd(const GsProblem& pr, const GsFwd& f, char* ws, hipStream_t s) {
    if (pr.B == 0 || pr.H == 0) return hipSuccess;
    GsArgs a = gs_args(pr, gs_plan(pr), f.x, f.g, f.lens, ws);
    a.first = f.h0;
    a.out = f.o;
    a.last = f.hT;
    a.states = f.states;
    return fwd_any(pr, a, s);
}

hipError_t launch_gated_scan_bwd(const GsProblem& pr, const GsBwd& f, char* ws, hipStream_t s) {
    if (pr.B == 0 || pr.H == 0) return hipSuccess;
    const GsPlan p = gs_plan(pr);
    const float* states = f.states;
    if (!states) {
        float* again = reinterpret_cast<float*>(ws + gs_ws(pr, 2).states);
        GsArgs a = gs_args(pr, p, f.x, f.g, f.lens, ws);
        a.first = f.h0;
        a.states = again;
        const hipError_t e = fwd_any(pr, a, s);
        if (e != hipSuccess) return e;
        states = again;
    }
    GsArgs a = gs_args(pr, p, f.x, f.g, f.lens, ws);
    a.y = f.dout;
    a.first = f.dhT;
    a.states_in = states;
    a.out = f.dx;
    a.dg = f.dg;
    a.last = f.dh0;
    return bwd_any(pr, a, s);
}

hipError_t launch_gated_scan_recurrent(const GsProblem& pr, const void* x, const float* g, float* state, void* o,
                                       hipStream_t s) {
    const long n = (long)pr.B * pr.H * pr.d;
    if (n * pr.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((n + 255) / 256)), block(256);
    prof_begin(s, "gated_scan_recurrent");
#define DN_GS_REC(E, C)                                                                                           \
    hipLaunchKernelGGL((gated_scan_recurrent_kernel<E, C>), grid, block, 0, s, static_cast<const E*>(x), g, state, \
                       static_cast<E*>(o), pr.B * pr.H, pr.T, pr.d)
    if (pr.bf16 && pr.coupled)
        DN_GS_REC(bf16, true);
    else if (pr.bf16)
        DN_GS_REC(bf16, false);
    else if (pr.coupled)
        DN_GS_REC(float, true);
    else
        DN_GS_REC(float, false);
#undef DN_GS_REC
    prof_end(s);
    return hipGetLastError();
}

}  // namespace dn
