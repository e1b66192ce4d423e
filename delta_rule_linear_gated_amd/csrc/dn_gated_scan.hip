// dn_gated_scan.hip -- gated linear recurrence, one state a channel:
//     h_t = e^{g_t} h_{t-1} + w_t x_t,   o_t = h_t,   w_t = 1 or (coupled) 1 - e^{g_t},
// its backward pass and its recurrent form.  Layouts as in include/dn.h.
//
// A step is the affine map h -> a h + b; a run of steps is the map {p, e}, p the product of
// its decays and e its end from a zero state.  A workgroup works on tiles: a run of steps of a
// strip of 64 channels (a lane each).  Each of its waves forms the map of its run of the tile
// in registers, the waves exchange the maps through LDS (one barrier), each takes its run's
// first state through the maps before it and goes over its registers again for the outputs.
// All of a tile's rows are loaded while the one before is worked on, and every tensor is
// read once.
//
// Enough strips: a workgroup walks the tiles of one strip, the state in a register.  Few
// strips (gs_plan): the tiles of all strips are handed out in the order of their steps, and a
// tile takes its first state from messages of the tiles before it in its strip (Chain).
//
// The backward goes from the last step with r_t = a_t D_t, the cotangent
// that leaves step t to earlier ones:
//     D_t = do_t + r_{t+1},   dx_t = w_t D_t,   dg_t = r_t (h_{t-1} - [coupled] x_t),
// h inside a tile from the state saved at its start.
#include <algorithm>

#include "dn_device.h"
#include "dn_gated_scan.h"
#include "dn_internal.h"

namespace dn {

namespace {

constexpr int kGsWaves = 16, kGsRun = 16;         // forward, marching: waves, steps of a wave in a tile
constexpr int kGsWavesC = 8, kGsRunC = 32;        // forward, chained
constexpr int kGsWavesB = 8;                      // backward: a tile begins at a saved state
constexpr int kGsRunB = kGsSaved / kGsWavesB;
constexpr int gs_tile(bool chain) { return chain ? kGsWavesC * kGsRunC : kGsWaves * kGsRun; }
constexpr int kGsUnits = 256;                     // compute units
static_assert(kGsSaved % kGsRun == 0 && kGsSaved % kGsRunC == 0, "saved states lie at the starts of runs");
constexpr int kRange = 0x7fffff00;                // bytes of a buffer range, at most
constexpr int kNowhere = 0x7ffffff0;              // an offset past every range: loads give zero, stores do nothing

struct GsArgs {
    int BH, H, T, d;
    int strips, tiles;           // tiles of a strip
    int reach;                   // a chained tile takes at most reach maps before its own
    int flat;                    // channel of a lane: 64 strip + lane of all, else of one head's row
    int NS;                      // saved states of a row
    const void *x, *y;           // y: dout
    const float* g;
    const int* lens;
    const float *first, *states_in;
    char* chain;                 // the next tile to hand out, then the messages (Chain)
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
        const unsigned n0 = 64u * strip, n = n0 + lane, row = n / a.d;   // 2^28 channels at most
        row0 = n0 / a.d;
        l.row = row;
        l.c = n - row * a.d;
        l.on = row < (unsigned)a.BH;
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

// Tiles of few strips: message `at` (the tile's place in the order in which they are handed
// out) holds the 64 lanes' maps, a word of p and e each, and their last states.  A word is valid
// by itself once it is not kUnset, to which a kernel sets all words before and which no value
// is written as, so that nothing but the word has to be ordered.  A tile's first state is the last
// state of the tile `reach` + 1 before it (or the strip's own), through the maps of the tiles
// between: those need no state, so that tiles in flight at once do not wait for one
// another's outputs.  The association depends on the tile alone, and so do the bits.
//
// Every wait ends: tiles are handed out in order by a counter, a workgroup finishes its own in
// that order, and a tile waits for earlier ones only, so that the earliest unfinished tile
// waits for nothing, however few workgroups run.
struct Chain {
    static constexpr int kEach = 16;   // maps that a wave gathers
    static constexpr unsigned kUnset = 0xffffffffu;   // a NaN
    static constexpr int kMessage = 64 * 8 + 64 * 4, kHead = 256;   // bytes

    static __device__ __forceinline__ char* message(const GsArgs& a, int at) { return a.chain + kHead + (long)at * kMessage; }
    static __device__ __forceinline__ unsigned long long* map_of(const GsArgs& a, int at) {
        return reinterpret_cast<unsigned long long*>(message(a, at)) + lane_id();
    }
    static __device__ __forceinline__ unsigned* last_of(const GsArgs& a, int at) {
        return reinterpret_cast<unsigned*>(message(a, at) + 64 * 8) + lane_id();
    }
    static __device__ __forceinline__ unsigned bits(float v) {   // any NaN as the quiet one
        return v == v ? __builtin_bit_cast(unsigned, v) : 0x7fc00000u;
    }
    static __device__ __forceinline__ void put_map(const GsArgs& a, int at, float p, float e) {
        __hip_atomic_store(map_of(a, at), (unsigned long long)bits(e) << 32 | bits(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    static __device__ __forceinline__ void put_last(const GsArgs& a, int at, float h) {
        __hip_atomic_store(last_of(a, at), bits(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    static __device__ __forceinline__ unsigned long long get_map(const GsArgs& a, int at) {
        return __hip_atomic_load(map_of(a, at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    static __device__ __forceinline__ unsigned get_last(const GsArgs& a, int at) {
        return __hip_atomic_load(last_of(a, at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }

    // The next tile (every lane of the wave gets it), -1: none is left.
    static __device__ __forceinline__ int claim(const GsArgs& a) {
        int n = 0;
        if (lane_id() == 0)
            n = (int)__hip_atomic_fetch_add(reinterpret_cast<unsigned*>(a.chain), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        n = __builtin_amdgcn_readfirstlane(n);
        return n < a.strips * a.tiles ? n : -1;
    }
    // Waves that gather: the first ones.
    static __device__ __forceinline__ int gatherers(const GsArgs& a) { return (a.reach + kEach - 1) / kEach; }
    // Wave w's share of what comes before tile `at`, k-th of its strip: a map, or (wave 0)
    // the state after its share, from the state before or from `first`.
    static __device__ __forceinline__ float2 gather(const GsArgs& a, int at, int k, int w, float first) {
        const int n = min(k, a.reach), lo = w * kEach, m = min(n - lo, kEach);   // m maps, oldest first
        float p = w == 0 ? 0.f : 1.f, e = 0.f;
        if (w == 0) {
            e = first;
            if (k > n) {
                const int from = at - (n + 1) * a.strips;
                unsigned u = get_last(a, from);
                while (!__all(u != kUnset)) {
                    __builtin_amdgcn_s_sleep(1);
                    u = get_last(a, from);
                }
                e = __builtin_bit_cast(float, u);
            }
        }
        constexpr int BATCH = 8;
        for (int i0 = 0; i0 < m; i0 += BATCH) {
            unsigned long long u[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) u[i] = get_map(a, at - (n - lo - min(i0 + i, m - 1)) * a.strips);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (i0 + i >= m) break;
                while (!__all((unsigned)u[i] != kUnset)) {
                    __builtin_amdgcn_s_sleep(1);
                    u[i] = get_map(a, at - (n - lo - (i0 + i)) * a.strips);
                }
                const float q = __builtin_bit_cast(float, (unsigned)u[i]);
                if (w > 0) p *= q;
                e = fmaf(q, e, __builtin_bit_cast(float, (unsigned)(u[i] >> 32)));
            }
        }
        return make_float2(p, e);
    }
};

// Forward.  Outputs, saved states and the last state, each where wanted.
template <typename T, bool COUPLED, bool CHAIN>
__global__ __launch_bounds__(64 * (CHAIN ? kGsWavesC : kGsWaves)) void gated_scan_fwd_kernel(GsArgs a) {
    constexpr int R = CHAIN ? kGsRunC : kGsRun, W = CHAIN ? kGsWavesC : kGsWaves, TILE = W * R;
    __shared__ float2 part[2][W][64], gathered[CHAIN ? W : 1][64];
    __shared__ int claimed[2];
    const int w = uniform_wave(), lane = lane_id();
    const int gatherers = CHAIN ? Chain::gatherers(a) : 0;
    int at = 0, next = CHAIN ? -1 : a.tiles > 1 ? 1 : -1, after = -1;
    if (CHAIN) {
        if (w == 0) at = Chain::claim(a);
        if (w == 0 && lane == 0) claimed[0] = at;
        __syncthreads();
        at = __builtin_amdgcn_readfirstlane(claimed[0]);
        if (at < 0) return;
        __syncthreads();
    } else if (a.tiles == 0) {
        at = -1;
    }
    long row0;
    Lane l = gs_lane(a, CHAIN ? at % a.strips : blockIdx.x, row0);
    float h = a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f;
    unsigned gn[R], xn[R];
    auto fetch = [&](const Lane& l, long row0, int t) {
        const bool full = __all(!l.on || l.len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, l.len, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, l.len, full);
    };
    auto prefetch = [&]() {   // the next tile's rows
        if (CHAIN) {
            long r;
            const Lane m = gs_lane(a, next % a.strips, r);
            fetch(m, r, next / a.strips * TILE + w * R);
        } else {
            fetch(l, row0, next * TILE + w * R);
        }
    };
    if (at >= 0) fetch(l, row0, (CHAIN ? at / a.strips : 0) * TILE + w * R);
    for (int buf = 0; at >= 0; buf ^= 1) {
        const int k = CHAIN ? at / a.strips : at, t = k * TILE + w * R;
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
        // a wave that gathers would wait for its rows with the messages: it loads them after
        bool ahead = next >= 0 && w >= gatherers;
        if (ahead) prefetch();
        part[buf][w][lane] = make_float2(gs_exp(sum), e);
        __syncthreads();
        if (CHAIN) {
            if (w == 0) {
                float p = 1.f, q = 0.f;
#pragma unroll
                for (int v = 0; v < W; ++v) {
                    const float2 m = part[buf][v][lane];
                    p *= m.x;
                    q = fmaf(m.x, q, m.y);
                }
                Chain::put_map(a, at, p, q);
            }
            if (w == W - 1) {   // tiles to work on after the next
                const int n = next < 0 ? Chain::claim(a) : -1, m = Chain::claim(a);
                if (lane == 0) claimed[0] = n, claimed[1] = m;
            }
            if (w < gatherers)
                gathered[w][lane] = Chain::gather(a, at, k, w, a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f);
            __syncthreads();
            h = gathered[0][lane].y;
            for (int v = 1; v < gatherers; ++v) h = fmaf(gathered[v][lane].x, h, gathered[v][lane].y);
            if (next < 0) next = __builtin_amdgcn_readfirstlane(claimed[0]);
            after = __builtin_amdgcn_readfirstlane(claimed[1]);
        } else {
            after = next >= 0 && next + 1 < a.tiles ? next + 1 : -1;
        }
        float mine = h;
#pragma unroll
        for (int v = 0; v < W; ++v) {
            const float2 m = part[buf][v][lane];
            if (v == w) mine = h;
            h = fmaf(m.x, h, m.y);
        }
        if (CHAIN && w == W - 1) Chain::put_last(a, at, h);
        if (CHAIN && !ahead && next >= 0) prefetch();
        if (a.states && l.on && t % kGsSaved == 0 && t < a.T) a.states[(l.row * a.NS + t / kGsSaved) * a.d + l.c] = mine;
        if (a.out) {
            const bool full = __all(!l.on || l.len >= t + R);
#pragma unroll
            for (int i = 0; i < R; ++i) b[i] = mine = fmaf(f[i], mine, b[i]);
            gs_store<T, R>(b, a.out, a, row0, l, t, l.len, full);
        }
        if (k == a.tiles - 1 && w == 0 && a.last && l.on) a.last[l.row * a.d + l.c] = h;
        at = next;
        next = after;
        if (CHAIN && at >= 0) l = gs_lane(a, at % a.strips, row0);
    }
    if (!CHAIN && a.tiles == 0 && a.last && w == 0 && l.on) a.last[l.row * a.d + l.c] = h;
}

// Backward: tiles from the last step on, k the number of tiles behind this one.
template <typename T, bool COUPLED, bool CHAIN>
__global__ __launch_bounds__(64 * kGsWavesB) void gated_scan_bwd_kernel(GsArgs a) {
    constexpr int R = kGsRunB, W = kGsWavesB;
    __shared__ float2 fore[2][W][64], back[2][W][64], gathered[CHAIN ? W : 1][64];
    __shared__ int claimed[2];
    const int w = uniform_wave(), lane = lane_id();
    const int gatherers = CHAIN ? Chain::gatherers(a) : 0;
    int at = 0, next = CHAIN ? -1 : a.tiles > 1 ? 1 : -1, after = -1;
    if (CHAIN) {
        if (w == 0) at = Chain::claim(a);
        if (w == 0 && lane == 0) claimed[0] = at;
        __syncthreads();
        at = __builtin_amdgcn_readfirstlane(claimed[0]);
        if (at < 0) return;
        __syncthreads();
    } else if (a.tiles == 0) {
        at = -1;
    }
    long row0;
    Lane l = gs_lane(a, CHAIN ? at % a.strips : blockIdx.x, row0);
    float r = a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f;
    unsigned gn[R], xn[R], yn[R];
    float hn = 0.f;
    auto fetch = [&](const Lane& l, long row0, int k) {
        const int t0 = (a.tiles - 1 - k) * kGsSaved, t = t0 + w * R;
        const bool full = __all(!l.on || l.len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, l.len, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, l.len, full);
        gs_load<T, R>(yn, a.y, a, row0, l, t, l.len, full);
        hn = l.len > t0 ? a.states_in[(l.row * a.NS + t0 / kGsSaved) * a.d + l.c] : 0.f;
    };
    auto prefetch = [&]() {
        if (CHAIN) {
            long r;
            const Lane m = gs_lane(a, next % a.strips, r);
            fetch(m, r, next / a.strips);
        } else {
            fetch(l, row0, next);
        }
    };
    if (at >= 0) fetch(l, row0, CHAIN ? at / a.strips : 0);
    for (int buf = 0; at >= 0; buf ^= 1) {
        const int k = CHAIN ? at / a.strips : at, t = (a.tiles - 1 - k) * kGsSaved + w * R;
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
        bool ahead = next >= 0 && w >= gatherers;
        if (ahead) prefetch();
#pragma unroll
        for (int i = R - 1; i >= 0; --i) q = f[i] * (q + y[i]);
        const float p = gs_exp(sum);
        fore[buf][w][lane] = make_float2(p, e);
        back[buf][w][lane] = make_float2(p, q);
        __syncthreads();
        if (CHAIN) {
            if (w == 0) {
                float p = 1.f, q = 0.f;
#pragma unroll
                for (int v = W - 1; v >= 0; --v) {
                    const float2 m = back[buf][v][lane];
                    p *= m.x;
                    q = fmaf(m.x, q, m.y);
                }
                Chain::put_map(a, at, p, q);
            }
            if (w == W - 1) {
                const int n = next < 0 ? Chain::claim(a) : -1, m = Chain::claim(a);
                if (lane == 0) claimed[0] = n, claimed[1] = m;
            }
            if (w < gatherers)
                gathered[w][lane] = Chain::gather(a, at, k, w, a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f);
            __syncthreads();
            r = gathered[0][lane].y;
            for (int v = 1; v < gatherers; ++v) r = fmaf(gathered[v][lane].x, r, gathered[v][lane].y);
            if (next < 0) next = __builtin_amdgcn_readfirstlane(claimed[0]);
            after = __builtin_amdgcn_readfirstlane(claimed[1]);
        } else {
            after = next >= 0 && next + 1 < a.tiles ? next + 1 : -1;
        }
        float mine = r;
#pragma unroll
        for (int v = W - 1; v >= 0; --v) {
            const float2 m = back[buf][v][lane];
            if (v == w) mine = r;
            r = fmaf(m.x, r, m.y);
        }
        if (CHAIN && w == W - 1) Chain::put_last(a, at, r);
        if (CHAIN && !ahead && next >= 0) prefetch();
#pragma unroll
        for (int v = 0; v < W - 1; ++v)
            if (v < w) {
                const float2 m = fore[buf][v][lane];
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
        const bool full = __all(!l.on || l.len >= t + R);
        gs_store<T, R>(x, a.out, a, row0, l, t, l.len, full);
        gs_store<float, R>(y, a.dg, a, row0, l, t, l.len, full);
        if (k == a.tiles - 1 && w == 0 && a.last && l.on) a.last[l.row * a.d + l.c] = r;
        at = next;
        next = after;
        if (CHAIN && at >= 0) l = gs_lane(a, at % a.strips, row0);
    }
    if (!CHAIN && a.tiles == 0 && a.last && w == 0 && l.on) a.last[l.row * a.d + l.c] = r;
}

// Before a chain: the counter is zero, every word of the messages unset.
__global__ __launch_bounds__(256) void gated_scan_clear_kernel(uint4* p, long n) {
    for (long i = blockIdx.x * 256L + threadIdx.x; i < n; i += gridDim.x * 256L) {
        const unsigned v = i < Chain::kHead / 16 ? 0u : Chain::kUnset;
        p[i] = make_uint4(v, v, v, v);
    }
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
    int flat, chain, tiles, reach;
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
GsPlan gs_plan(const GsProblem& pr, bool bwd) {
    GsPlan p{};
    gs_strips(pr, &p);
    p.chain = p.strips > 0 && p.strips < kGsUnits && pr.T > 2 * (bwd ? kGsSaved : gs_tile(true));
    const int tile = bwd ? kGsSaved : gs_tile(p.chain);
    p.tiles = (int)(((long)pr.T + tile - 1) / tile);
    // the tiles of a strip that are in flight at once
    if (p.chain) p.reach = (int)std::min<long>((bwd ? kGsWavesB : kGsWavesC) * Chain::kEach, std::max<long>(4, kGsUnits / p.strips));
    return p;
}

size_t gs_chain_bytes(const GsPlan& p) { return p.chain ? Chain::kHead + (size_t)p.strips * p.tiles * Chain::kMessage : 0; }

struct GsWs {
    size_t states, total;   // the messages lie at the start
};
GsWs gs_ws(const GsProblem& pr, int pass) {
    GsWs w{};
    if (pass != 1) w.states = gs_chain_bytes(gs_plan(pr, false));
    if (pass != 0) w.states = std::max(w.states, gs_chain_bytes(gs_plan(pr, true)));
    w.states = al256(w.states);
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
    a.tiles = p.tiles;
    a.reach = p.reach;
    a.flat = p.flat;
    a.NS = (int)(((long)pr.T + kGsSaved - 1) / kGsSaved);
    a.x = x;
    a.g = g;
    a.lens = lens;
    a.chain = ws;
    return a;
}

hipError_t clear_chain(const GsPlan& p, char* ws, hipStream_t s) {
    const long n = (long)(gs_chain_bytes(p) / 16);
    prof_begin(s, "gated_scan_clear");
    hipLaunchKernelGGL(gated_scan_clear_kernel, dim3((unsigned)std::min<long>((n + 255) / 256, 4 * kGsUnits)), dim3(256), 0, s,
                       reinterpret_cast<uint4*>(ws), n);
    prof_end(s);
    return hipGetLastError();
}
unsigned gs_grid(const GsPlan& p) { return (unsigned)(p.chain ? std::min<long>(p.strips * p.tiles, kGsUnits) : p.strips); }

template <typename T, bool COUPLED> hipError_t fwd_launch(const GsPlan& p, const GsArgs& a, hipStream_t s) {
    const dim3 grid(gs_grid(p)), block(64 * (p.chain ? kGsWavesC : kGsWaves));
    prof_begin(s, "gated_scan_fwd");
    if (p.chain)
        hipLaunchKernelGGL((gated_scan_fwd_kernel<T, COUPLED, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((gated_scan_fwd_kernel<T, COUPLED, false>), grid, block, 0, s, a);
    prof_end(s);
    return hipGetLastError();
}
template <typename T, bool COUPLED> hipError_t bwd_launch(const GsPlan& p, const GsArgs& a, hipStream_t s) {
    const dim3 grid(gs_grid(p)), block(64 * kGsWavesB);
    prof_begin(s, "gated_scan_bwd");
    if (p.chain)
        hipLaunchKernelGGL((gated_scan_bwd_kernel<T, COUPLED, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((gated_scan_bwd_kernel<T, COUPLED, false>), grid, block, 0, s, a);
    prof_end(s);
    return hipGetLastError();
}
hipError_t fwd_any(const GsProblem& pr, const GsPlan& p, const GsArgs& a, hipStream_t s) {
    if (p.chain) {
        const hipError_t e = clear_chain(p, a.chain, s);
        if (e != hipSuccess) return e;
    }
    if (pr.bf16) return pr.coupled ? fwd_launch<bf16, true>(p, a, s) : fwd_launch<bf16, false>(p, a, s);
    return pr.coupled ? fwd_launch<float, true>(p, a, s) : fwd_launch<float, false>(p, a, s);
}
hipError_t bwd_any(const GsProblem& pr, const GsPlan& p, const GsArgs& a, hipStream_t s) {
    if (p.chain) {
        const hipError_t e = clear_chain(p, a.chain, s);
        if (e != hipSuccess) return e;
    }
    if (pr.bf16) return pr.coupled ? bwd_launch<bf16, true>(p, a, s) : bwd_launch<bf16, false>(p, a, s);
    return pr.coupled ? bwd_launch<float, true>(p, a, s) : bwd_launch<float, false>(p, a, s);
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
    const GsPlan p = gs_plan(pr, false);
    GsArgs a = gs_args(pr, p, f.x, f.g, f.lens, ws);
    a.first = f.h0;
    a.out = f.o;
    a.last = f.hT;
    a.states = f.states;
    return fwd_any(pr, p, a, s);
}

hipError_t launch_gated_scan_bwd(const GsProblem& pr, const GsBwd& f, char* ws, hipStream_t s) {
    if (pr.B == 0 || pr.H == 0) return hipSuccess;
    const float* states = f.states;
    if (!states && pr.T > 0) {
        float* again = reinterpret_cast<float*>(ws + gs_ws(pr, 2).states);
        const GsPlan p = gs_plan(pr, false);
        GsArgs a = gs_args(pr, p, f.x, f.g, f.lens, ws);
        a.first = f.h0;
        a.states = again;
        const hipError_t e = fwd_any(pr, p, a, s);
        if (e != hipSuccess) return e;
        states = again;
    }
    const GsPlan p = gs_plan(pr, true);
    GsArgs a = gs_args(pr, p, f.x, f.g, f.lens, ws);
    a.y = f.dout;
    a.first = f.dhT;
    a.states_in = states;
    a.out = f.dx;
    a.dg = f.dg;
    a.last = f.dh0;
    return bwd_any(pr, p, a, s);
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
