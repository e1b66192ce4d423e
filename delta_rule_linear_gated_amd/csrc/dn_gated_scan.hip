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
// read once: the bytes bound it (8 x 16 heads of 128, 4096 steps, bf16: forward 114 us, backward
// 200, 4.7 TB/s both; a large copy runs at 5.1).
//
// Times here and at gs_plan are of calls in a captured graph, clearing included, on inputs that no
// cache holds.  In a training step the backward finds part of the forward's inputs in the last-level
// cache: the two of this case take 292 together, and a trace of them shows 120 and 176.
//
// Marching, a workgroup walks the tiles of one strip, the state in a register.  Where the strips
// do not fill the chip (gs_plan), the tiles of all strips are handed out in the order of their
// steps, and a tile takes its first state from messages of the tiles before it in its strip (Chain).
//
// The backward goes from the last step with r_t = a_t D_t, the cotangent
// that leaves step t to earlier ones:
//     D_t = do_t + r_{t+1},   dx_t = w_t D_t,   dg_t = r_t (h_{t-1} - [coupled] x_t),
// h inside a tile from the state saved at its start.
#include <algorithm>

#include "dn_device.h"
#include "dn_gated_scan_plan.h"
#include "dn_internal.h"
#include "dn_wait.h"

namespace dn {

namespace {

static_assert(kGsXcds == kXcds, "one count of the dies");
constexpr int kNowhere = 0x7ffffff0;              // an offset past every range: loads give zero, stores do nothing

struct GsArgs {
    int BH, H, T, d;
    int strips, tiles;           // tiles of a strip
    int reach;                   // a chained tile takes at most reach maps before its own
    int flat;                    // strips of the channels of all heads in a row, else of one head's
    int NS;                      // saved states of a row
    const void *x, *y;           // y: dout
    const float* g;
    const int* lens;
    const float *first, *states_in;
    char* chain;                 // the next tile to hand out, then the messages (Chain)
    void* out;                   // o or dx; NULL: not wanted
    float *dg, *last, *states;
};

// A lane's channel and steps: a strip is 64 / G channels, and a wave's lanes take G runs of R
// steps of each, one after the other.
struct Lane {
    long row;      // (b, h)
    int c, off;    // channel; elements from the wave's first step of the strip's first row to the lane's
    int ahead;     // steps from the wave's first to the lane's
    int len;       // steps of its sequence, 0 for an idle lane
    bool on;
};
template <int G, int R>
__device__ __forceinline__ Lane gs_lane(const GsArgs& a, int strip, long& row0, const int* len = nullptr) {   // len: known
    constexpr int C = 64 / G;
    Lane l;
    const int lane = lane_id() % C;
    if (a.flat) {
        const unsigned n0 = (unsigned)C * strip, n = n0 + lane, row = n / a.d;   // 2^28 channels at most
        row0 = n0 / a.d;
        l.row = row;
        l.c = n - row * a.d;
        l.on = row < (unsigned)a.BH;
    } else {
        const int per = (a.d + C - 1) / C;
        row0 = l.row = strip / per;
        l.c = strip % per * C + lane;
        l.on = l.c < a.d;
    }
    l.ahead = lane_id() / C * R;
    l.off = l.on ? (int)(((unsigned)(l.row - row0) * a.T + l.ahead) * a.d + l.c) : 0;
    l.len = len ? *len : !l.on ? 0 : a.lens ? min(max(a.lens[l.row / a.H], 0), a.T) : a.T;
    return l;
}
// Strips marched by a workgroup each: the G strips of 64 channels go to one XCD (workgroups go
// to the XCDs in turn), whose L2 then reads each line once for all of them.
template <int G> __device__ __forceinline__ int gs_strip() {
    const int x = blockIdx.x % kXcds, j = blockIdx.x / kXcds;
    return (j / G * kXcds + x) * G + j % G;
}

// What lies from element `at` on of a tensor of n elements, as a buffer.
template <typename T> __device__ __forceinline__ __amdgpu_buffer_rsrc_t gs_range(const void* p, long n, long at) {
    const long left = (n - at) * (long)sizeof(T);
    const int bytes = left <= 0 ? 0 : left < kGsRange ? (int)left : kGsRange;
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

// A lane's R rows, a step's value in a register; t: the wave's first step.  Rows past a lane's
// length read as zero (g: a factor of one) and are written as zero.  All of a wave's lanes full
// (the wave asks with __all): the steps are scalar offsets, else selects.
template <typename T, int R>
__device__ __forceinline__ void gs_load(unsigned (&v)[R], const void* p, const GsArgs& a, long row0, const Lane& l, int t,
                                        bool full) {
    const long n = (long)a.BH * a.T * a.d, at = (row0 * a.T + t) * a.d;
    const auto r = gs_range<T>(p, n, at);
    const int step = a.d * (int)sizeof(T), off = l.on ? (int)((unsigned)l.off * (unsigned)sizeof(T)) : kNowhere;
    if (full) {
#pragma unroll
        for (int i = 0; i < R; ++i) v[i] = Bits<T>::load(r, off, i * step);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            v[i] = Bits<T>::load(r, t + l.ahead + i < l.len ? (int)((unsigned)off + (unsigned)(i * step)) : kNowhere, 0);
    }
}
template <typename T, int R>
__device__ __forceinline__ void gs_store(const float (&v)[R], void* p, const GsArgs& a, long row0, const Lane& l, int t,
                                         bool full) {
    const long n = (long)a.BH * a.T * a.d, at = (row0 * a.T + t) * a.d;
    const auto r = gs_range<T>(p, n, at);
    const int step = a.d * (int)sizeof(T), off = l.on ? (int)((unsigned)l.off * (unsigned)sizeof(T)) : kNowhere;
    if (full) {
#pragma unroll
        for (int i = 0; i < R; ++i) Bits<T>::store(v[i], r, off, i * step);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int s = t + l.ahead + i;
            Bits<T>::store(s < l.len ? v[i] : 0.f, r, l.on && s < a.T ? (int)((unsigned)off + (unsigned)(i * step)) : kNowhere,
                           0);
        }
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

// Maps of a wave's runs: {p, e} of a lane's run becomes that of all of its channel's runs up to
// and with it (REV: from it on), and `out` the map of the runs before (REV: behind) it.
template <int G, bool REV> __device__ __forceinline__ void gs_join(float& p, float& e, float2& out) {
    constexpr int C = 64 / G;
    const int l = lane_id();
#pragma unroll
    for (int s = C; s < 64; s *= 2) {
        const float q = REV ? __shfl_down(p, s) : __shfl_up(p, s), f = REV ? __shfl_down(e, s) : __shfl_up(e, s);
        if (REV ? l + s < 64 : l >= s) {
            e = fmaf(p, f, e);
            p *= q;
        }
    }
    out = make_float2(1.f, 0.f);
    if (G > 1) {
        const float q = REV ? __shfl_down(p, C) : __shfl_up(p, C), f = REV ? __shfl_down(e, C) : __shfl_up(e, C);
        if (REV ? l + C < 64 : l >= C) out = make_float2(q, f);
    }
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
// Every message comes: tiles are handed out in order by a counter, a workgroup finishes its own in
// that order, and a tile waits for earlier ones only, so that the earliest unfinished tile
// waits for nothing, however few workgroups run.  That holds while nobody else writes to the
// workspace; where somebody does (two calls on it that are not ordered), messages may be wiped
// out for good.  So a wave stops looking at a word after kLooks looks, 0.14 s (a tile takes 5 us),
// and goes on with a NaN in its place.  A message concerns the next reach + 1 tiles of its strip
// alone, a few of each workgroup, which wait for nine words each at most, and those that they keep
// waiting: the launch ends within seconds.  (A count of its own for each word costs up to 2 %: 16
// heads of 128, 32768 steps, a call that saves no states 127.2 -> 129.5 us; one count kept over the
// tiles, in a register or in LDS, made the bf16 forward 4 % slower.)
struct Chain {
    static constexpr int kEach = kGsEach;
    static constexpr int kLooks = 1 << 20;
    static constexpr unsigned kUnset = 0xffffffffu, kNan = 0x7fc00000u;   // a NaN that no value is written as; the one that NaNs are
    static constexpr int kMessage = kGsMessage, kHead = kGsHead;   // bytes

    static __device__ __forceinline__ char* message(const GsArgs& a, int at) { return a.chain + kHead + (long)at * kMessage; }
    static __device__ __forceinline__ unsigned long long* map_of(const GsArgs& a, int at) {
        return reinterpret_cast<unsigned long long*>(message(a, at)) + lane_id();
    }
    static __device__ __forceinline__ unsigned* last_of(const GsArgs& a, int at) {
        return reinterpret_cast<unsigned*>(message(a, at) + 64 * 8) + lane_id();
    }
    static __device__ __forceinline__ unsigned bits(float v) {   // any NaN as the quiet one
        return v == v ? __builtin_bit_cast(unsigned, v) : kNan;
    }
    static __device__ __forceinline__ void put_map(const GsArgs& a, int at, float2 m) {
        __hip_atomic_store(map_of(a, at), (unsigned long long)bits(m.y) << 32 | bits(m.x), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
    // A workgroup's first tile; slot: LDS.
    static __device__ __forceinline__ int first(const GsArgs& a, int* slot) {
        if (wave_id() == 0) {
            const int n = claim(a);
            if (lane_id() == 0) *slot = n;
        }
        __syncthreads();
        const int n = __builtin_amdgcn_readfirstlane(*slot);
        __syncthreads();
        return n;
    }
    static __device__ __forceinline__ float2 then(float2 m, float2 n) { return make_float2(n.x * m.x, fmaf(n.x, m.y, n.y)); }
    // Waves that gather: the first ones.
    static __device__ __forceinline__ int gatherers(const GsArgs& a) { return (a.reach + kEach - 1) / kEach; }
    // Wave w's share of what comes before tile `at`: a map, or (wave 0) the state after its share,
    // from the state before it or the strip's own.  Asked for early, so that the answers are
    // there when the rows that were on their way before are (loads come back in order).
    struct Wave {
        unsigned long long u[kEach];
        unsigned base;
        float first;

        __device__ __forceinline__ void share(const GsArgs& a, int at, int w, int& k, int& n, int& m) const {
            k = at / a.strips;
            n = min(k, a.reach);
            m = min(n - w * kEach, kEach);   // maps, oldest first
        }
        __device__ __forceinline__ void ask(const GsArgs& a, int at, int w) {
            int k, n, m;
            share(a, at, w, k, n, m);
            first = 0.f;
            base = 0;
            if (w == 0 && k > n) base = get_last(a, at - (n + 1) * a.strips);
            if (w == 0 && k <= n && a.first) {
                long row0;
                const Lane l = gs_lane<1, 1>(a, at % a.strips, row0, &k);   // its length does not matter
                if (l.on) first = a.first[l.row * a.d + l.c];
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i < m) u[i] = get_map(a, at - (n - w * kEach - i) * a.strips);
        }
        __device__ __forceinline__ float2 answer(const GsArgs& a, int at, int w) {
            int k, n, m;
            share(a, at, w, k, n, m);
            float p = w == 0 ? 0.f : 1.f, e = first;
            if (w == 0 && k > n) {
                wait_until([&] { return __all(base != kUnset); },
                           [&] {
                               __builtin_amdgcn_s_sleep(1);
                               base = get_last(a, at - (n + 1) * a.strips);
                           },
                           [&] { base = kNan; }, kLooks);
                e = __builtin_bit_cast(float, base);
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (i >= m) break;
                wait_until([&] { return __all((unsigned)u[i] != kUnset); },
                           [&] {
                               __builtin_amdgcn_s_sleep(1);
                               u[i] = get_map(a, at - (n - w * kEach - i) * a.strips);
                           },
                           [&] { u[i] = (unsigned long long)kNan << 32 | kNan; }, kLooks);
                const float q = __builtin_bit_cast(float, (unsigned)u[i]);
                if (w > 0) p *= q;
                e = fmaf(q, e, __builtin_bit_cast(float, (unsigned)(u[i] >> 32)));
            }
            return make_float2(p, e);
        }
    };
};

// Forward, marching.  Outputs, saved states and the last state, each where wanted.  Four waves a SIMD
// leave 128 registers; bf16 with two or four runs a wave (coupled) or four or eight (not) spills two.
template <typename T, bool COUPLED, int W, int G>
__global__ __launch_bounds__(64 * W, 4) void gated_scan_fwd_kernel(GsArgs a) {
    constexpr int R = kGsRun, TILE = W * G * R, C = 64 / G;
    __shared__ float2 part[2][W][C];
    const int w = uniform_wave(), lane = lane_id(), c = lane % C, strip = gs_strip<G>();
    if (strip >= a.strips) return;
    long row0;
    const Lane l = gs_lane<G, R>(a, strip, row0);
    float h = a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f;
    unsigned gn[R], xn[R];
    auto fetch = [&](int t) {
        const bool full = __all(!l.on || l.len >= t + l.ahead + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, full);
    };
    if (a.tiles > 0) fetch(w * G * R);
    for (int k = 0; k < a.tiles; ++k) {
        const int t = k * TILE + w * G * R, tl = t + l.ahead;
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
        if (k + 1 < a.tiles) fetch(t + TILE);
        float p = gs_exp(sum);
        float2 own;
        gs_join<G, false>(p, e, own);
        if (lane >= 64 - C) part[k & 1][w][c] = make_float2(p, e);
        __syncthreads();
        float mine = h;
#pragma unroll
        for (int v = 0; v < W; ++v) {
            const float2 m = part[k & 1][v][c];
            if (v == w) mine = h;
            h = fmaf(m.x, h, m.y);
        }
        if (G > 1) mine = fmaf(own.x, mine, own.y);
        if (a.states && l.on && tl % kGsSaved == 0 && tl < a.T) a.states[(l.row * a.NS + tl / kGsSaved) * a.d + l.c] = mine;
        if (!a.out) continue;
        const bool full = __all(!l.on || l.len >= tl + R);
#pragma unroll
        for (int i = 0; i < R; ++i) b[i] = mine = fmaf(f[i], mine, b[i]);
        gs_store<T, R>(b, a.out, a, row0, l, t, full);
    }
    if (a.last && w == 0 && lane < C && l.on) a.last[l.row * a.d + l.c] = h;
}

// Forward, chained: outputs are a tile behind the maps, so that a tile's map has been on its
// way to the others for as long as a tile takes when they ask for it (32 strips, 32768 steps, bf16:
// 131 us, 4.1 TB/s; outputs at once, as it was first, 168).  12 waves: as many as have the registers of
// two tiles, 168 each (bf16 157 and 159; fp32 all, and coupled it spills six; 24 to 39 scalars lie in
// vector registers' lanes).
template <typename T, bool COUPLED> __global__ __launch_bounds__(64 * kGsWavesC) void gated_scan_fwd_chain_kernel(GsArgs a) {
    constexpr int R = kGsRun, W = kGsWavesC, TILE = W * R;
    __shared__ float2 part[2][W][64], gathered[2][W][64];
    __shared__ int claimed[2][2];
    const int w = uniform_wave(), lane = lane_id(), gatherers = Chain::gatherers(a);
    // tiles: outputs to write, map to form (its rows on the way), rows to load
    int cur = -1, nxt = Chain::first(a, &claimed[1][0]), nx2 = -1;
    if (nxt < 0) return;
    unsigned gn[R], xn[R];
    int len0 = 0, len1 = 0, len2 = 0;   // lengths of the lanes of cur, nxt, nx2
    auto fetch = [&](int at, int& len) {
        long row0;
        const Lane l = gs_lane<1, R>(a, at % a.strips, row0);
        const int t = at / a.strips * TILE + w * R;
        const bool full = __all(!l.on || l.len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, full);
        len = l.len;
    };
    fetch(nxt, len1);
    float f0[R], b0[R];
    float2 before0 = make_float2(1.f, 0.f), all0 = before0;   // cur's maps: of the waves before this one; whole (last wave)
    for (int n = 0; cur >= 0 || nxt >= 0; ++n) {
        const int buf = n & 1;
        Chain::Wave in;
        if (cur >= 0 && w < gatherers) in.ask(a, cur, w);
        int c0 = -1, c1 = -1;
        if (w == W - 1) {
            if (n == 0) c0 = Chain::claim(a);
            if (n == 0 || nx2 >= 0) c1 = Chain::claim(a);
        }
        float f1[R], b1[R], sum = 0.f, e = 0.f;
        if (nxt >= 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float g = Bits<float>::value(gn[i]);
                b1[i] = Bits<T>::value(xn[i]);
                f1[i] = gs_exp(g);
                if (COUPLED) b1[i] *= gs_rest(g, f1[i]);
                sum += g;
                e = fmaf(f1[i], e, b1[i]);
            }
            part[buf][w][lane] = make_float2(gs_exp(sum), e);
        }
        if (cur >= 0 && w < gatherers) gathered[buf][w][lane] = in.answer(a, cur, w);
        const bool fetched = nx2 >= 0;
        if (fetched) fetch(nx2, len2);
        if (w == W - 1 && lane == 0) claimed[buf][0] = c0, claimed[buf][1] = c1;
        __syncthreads();
        if (n == 0) nx2 = __builtin_amdgcn_readfirstlane(claimed[buf][0]);
        const int nx3 = __builtin_amdgcn_readfirstlane(claimed[buf][1]);
        if (!fetched && nx2 >= 0) fetch(nx2, len2);
        float2 before1 = make_float2(1.f, 0.f), all1 = before1;
        if (nxt >= 0) {
            for (int v = 0; v < w; ++v) before1 = Chain::then(before1, part[buf][v][lane]);
            if (w == W - 1) {
                all1 = Chain::then(before1, part[buf][w][lane]);
                Chain::put_map(a, nxt, all1);
            }
        }
        if (cur >= 0) {
            float h = gathered[buf][0][lane].y;
            for (int v = 1; v < gatherers; ++v) h = fmaf(gathered[buf][v][lane].x, h, gathered[buf][v][lane].y);
            long row0;
            const Lane l = gs_lane<1, R>(a, cur % a.strips, row0, &len0);
            const int k = cur / a.strips, t = k * TILE + w * R;
            if (w == W - 1) {
                const float last = fmaf(all0.x, h, all0.y);
                Chain::put_last(a, cur, last);
                if (k == a.tiles - 1 && a.last && l.on) a.last[l.row * a.d + l.c] = last;
            }
            h = fmaf(before0.x, h, before0.y);
            if (a.states && l.on && t % kGsSaved == 0 && t < a.T) a.states[(l.row * a.NS + t / kGsSaved) * a.d + l.c] = h;
            if (a.out) {
                const bool full = __all(!l.on || l.len >= t + R);
#pragma unroll
                for (int i = 0; i < R; ++i) b0[i] = h = fmaf(f0[i], h, b0[i]);
                gs_store<T, R>(b0, a.out, a, row0, l, t, full);
            }
        }
        cur = nxt, nxt = nx2, nx2 = nx3;
        len0 = len1, len1 = len2;
        before0 = before1, all0 = all1;
#pragma unroll
        for (int i = 0; i < R; ++i) f0[i] = f1[i], b0[i] = b1[i];
    }
}

// Backward, marching from the last step; k: tiles behind this one.
template <typename T, bool COUPLED, int W, int G>
__global__ __launch_bounds__(64 * W, 2) void gated_scan_bwd_kernel(GsArgs a) {
    constexpr int R = kGsRunB, TILE = W * G * R, C = 64 / G;
    constexpr int SHARE = W < kGsWavesB ? W : W / G;   // waves on the steps of one saved state (fewer waves: one tile, of the first)
    __shared__ float2 fore[2][W][C], back[2][W][C];
    const int w = uniform_wave(), lane = lane_id(), c = lane % C, strip = gs_strip<G>();
    if (strip >= a.strips) return;
    long row0;
    const Lane l = gs_lane<G, R>(a, strip, row0);
    float r = a.first && l.on ? a.first[l.row * a.d + l.c] : 0.f;
    unsigned gn[R], xn[R], yn[R];
    float hn = 0.f;
    auto fetch = [&](int t) {
        const int saved = t / kGsSaved;
        const bool full = __all(!l.on || l.len >= t + l.ahead + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, full);
        gs_load<T, R>(yn, a.y, a, row0, l, t, full);
        hn = l.len > saved * kGsSaved ? a.states_in[(l.row * a.NS + saved) * a.d + l.c] : 0.f;
    };
    if (a.tiles > 0) fetch((a.tiles - 1) * TILE + w * G * R);
    for (int k = 0; k < a.tiles; ++k) {
        const int t = (a.tiles - 1 - k) * TILE + w * G * R;
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
        if (k + 1 < a.tiles) fetch(t - TILE);
#pragma unroll
        for (int i = R - 1; i >= 0; --i) q = f[i] * (q + y[i]);
        float p = gs_exp(sum), pr = p;
        float2 own, ownr;
        gs_join<G, false>(p, e, own);
        gs_join<G, true>(pr, q, ownr);
        if (SHARE > 1 && lane >= 64 - C) fore[k & 1][w][c] = make_float2(p, e);
        if (lane < C) back[k & 1][w][c] = make_float2(pr, q);
        __syncthreads();
        float mine = r;
#pragma unroll
        for (int v = W - 1; v >= 0; --v) {
            const float2 m = back[k & 1][v][c];
            if (v == w) mine = r;
            r = fmaf(m.x, r, m.y);
        }
        if (G > 1) mine = fmaf(ownr.x, mine, ownr.y);
#pragma unroll
        for (int v = 0; v < SHARE - 1; ++v)
            if (v < w % SHARE) {
                const float2 m = fore[k & 1][w / SHARE * SHARE + v][c];
                h = fmaf(m.x, h, m.y);
            }
        if (G > 1) h = fmaf(own.x, h, own.y);
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
        const bool full = __all(!l.on || l.len >= t + l.ahead + R);
        gs_store<T, R>(x, a.out, a, row0, l, t, full);
        gs_store<float, R>(y, a.dg, a, row0, l, t, full);
    }
    if (a.last && w == 0 && lane < C && l.on) a.last[l.row * a.d + l.c] = r;
}

// Backward, chained from the last tile of every strip; results are a tile behind the maps.  The
// states inside a tile come from the saved one at its start and wait for no other tile (32 strips,
// 32768 steps, bf16: 206 us, 4.6 TB/s; results at once, as it was first, 250).
template <typename T, bool COUPLED> __global__ __launch_bounds__(64 * kGsWavesB) void gated_scan_bwd_chain_kernel(GsArgs a) {
    constexpr int R = kGsRunB, W = kGsWavesB, TILE = W * R;
    static_assert(TILE == kGsSaved, "a tile begins at a saved state");
    __shared__ float2 fore[2][W][64], back[2][W][64], gathered[2][W][64];
    __shared__ int claimed[2][2];
    const int w = uniform_wave(), lane = lane_id(), gatherers = Chain::gatherers(a);
    int cur = -1, nxt = Chain::first(a, &claimed[1][0]), nx2 = -1;
    if (nxt < 0) return;
    unsigned gn[R], xn[R], yn[R];
    float hn = 0.f;
    int len0 = 0, len1 = 0, len2 = 0;
    auto fetch = [&](int at, int& len) {
        long row0;
        const Lane l = gs_lane<1, R>(a, at % a.strips, row0);
        const int saved = a.tiles - 1 - at / a.strips, t = saved * TILE + w * R;
        const bool full = __all(!l.on || l.len >= t + R);
        gs_load<float, R>(gn, a.g, a, row0, l, t, full);
        gs_load<T, R>(xn, a.x, a, row0, l, t, full);
        gs_load<T, R>(yn, a.y, a, row0, l, t, full);
        hn = l.len > saved * TILE ? a.states_in[(l.row * a.NS + saved) * a.d + l.c] : 0.f;
        len = l.len;
    };
    fetch(nxt, len1);
    float f0[R], w0[R], y0[R], s0[R];   // s: h_{t-1}, less x_t if coupled
    float2 behind0 = make_float2(1.f, 0.f), all0 = behind0;   // cur's maps: of the waves behind this one; whole (wave 0)
    for (int n = 0; cur >= 0 || nxt >= 0; ++n) {
        const int buf = n & 1;
        Chain::Wave in;
        if (cur >= 0 && w < gatherers) in.ask(a, cur, w);
        int c0 = -1, c1 = -1;
        if (w == W - 1) {
            if (n == 0) c0 = Chain::claim(a);
            if (n == 0 || nx2 >= 0) c1 = Chain::claim(a);
        }
        float f1[R], w1[R], y1[R], s1[R], h = 0.f;
        if (nxt >= 0) {
            float sum = 0.f, e = 0.f, q = 0.f;
            h = hn;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float g = Bits<float>::value(gn[i]);
                s1[i] = Bits<T>::value(xn[i]);
                y1[i] = Bits<T>::value(yn[i]);
                f1[i] = gs_exp(g);
                w1[i] = COUPLED ? gs_rest(g, f1[i]) : 1.f;
                sum += g;
                e = fmaf(f1[i], e, w1[i] * s1[i]);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) q = f1[i] * (q + y1[i]);
            const float p = gs_exp(sum);
            fore[buf][w][lane] = make_float2(p, e);
            back[buf][w][lane] = make_float2(p, q);
        }
        if (cur >= 0 && w < gatherers) gathered[buf][w][lane] = in.answer(a, cur, w);
        const bool fetched = nx2 >= 0;
        if (fetched) fetch(nx2, len2);
        if (w == W - 1 && lane == 0) claimed[buf][0] = c0, claimed[buf][1] = c1;
        __syncthreads();
        if (n == 0) nx2 = __builtin_amdgcn_readfirstlane(claimed[buf][0]);
        const int nx3 = __builtin_amdgcn_readfirstlane(claimed[buf][1]);
        if (!fetched && nx2 >= 0) fetch(nx2, len2);
        float2 behind1 = make_float2(1.f, 0.f), all1 = behind1;
        if (nxt >= 0) {
            for (int v = W - 1; v > w; --v) behind1 = Chain::then(behind1, back[buf][v][lane]);
            if (w == 0) {
                all1 = Chain::then(behind1, back[buf][w][lane]);
                Chain::put_map(a, nxt, all1);
            }
            for (int v = 0; v < w; ++v) h = fmaf(fore[buf][v][lane].x, h, fore[buf][v][lane].y);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float x = s1[i];
                s1[i] = COUPLED ? h - x : h;
                h = fmaf(f1[i], h, w1[i] * x);
            }
        }
        if (cur >= 0) {
            float r = gathered[buf][0][lane].y;
            for (int v = 1; v < gatherers; ++v) r = fmaf(gathered[buf][v][lane].x, r, gathered[buf][v][lane].y);
            long row0;
            const Lane l = gs_lane<1, R>(a, cur % a.strips, row0, &len0);
            const int k = cur / a.strips, t = (a.tiles - 1 - k) * TILE + w * R;
            if (w == 0) {
                const float last = fmaf(all0.x, r, all0.y);
                Chain::put_last(a, cur, last);
                if (k == a.tiles - 1 && a.last && l.on) a.last[l.row * a.d + l.c] = last;
            }
            r = fmaf(behind0.x, r, behind0.y);
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const float D = y0[i] + r;
                r = f0[i] * D;
                y0[i] = COUPLED ? w0[i] * D : D;
                s0[i] *= r;
            }
            const bool full = __all(!l.on || l.len >= t + R);
            gs_store<T, R>(y0, a.out, a, row0, l, t, full);
            gs_store<float, R>(s0, a.dg, a, row0, l, t, full);
        }
        cur = nxt, nxt = nx2, nx2 = nx3;
        len0 = len1, len1 = len2;
        behind0 = behind1, all0 = all1;
#pragma unroll
        for (int i = 0; i < R; ++i) f0[i] = f1[i], w0[i] = w1[i], y0[i] = y1[i], s0[i] = s1[i];
    }
}

// Before a chain: the counter stands at the first tile, every word of the messages is unset.
__global__ __launch_bounds__(256) void gated_scan_clear_kernel(uint4* p, long n, int first_tile) {
    for (long i = blockIdx.x * 256L + threadIdx.x; i < n; i += gridDim.x * 256L) {
        const unsigned v = i < Chain::kHead / 16 ? 0u : Chain::kUnset;
        p[i] = make_uint4(i == 0 ? first_tile : v, v, v, v);
    }
}

// Recurrent form: a thread a channel, the state in a register over the steps; the latency of
// its few rows is all there is to it (131072 channels, one step, bf16: 2.4 us).
template <typename T, bool COUPLED>
__global__ __launch_bounds__(256) void gated_scan_recurrent_kernel(const T* x, const float* g, float* state, T* o, int BH,
                                                                   int steps, int d) {
    const unsigned n = blockIdx.x * 256u + threadIdx.x, row = n / d;   // 2^28 channels at most
    if (row >= (unsigned)BH) return;
    const long at = (long)row * steps * d + (n - row * d);
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

hipError_t clear_chain(const GsPlan& p, char* ws, int first_tile, hipStream_t s) {
    const long n = (long)(gs_chain_bytes(p) / 16);
    prof_begin(s, "gated_scan_clear");
    hipLaunchKernelGGL(gated_scan_clear_kernel, dim3((unsigned)std::min<long>((n + 255) / 256, 4 * kGsUnits)), dim3(256), 0, s,
                       reinterpret_cast<uint4*>(ws), n, first_tile);
    prof_end(s);
    return hipGetLastError();
}
unsigned gs_grid(const GsPlan& p) {
    return (unsigned)(p.chain ? std::min<long>(p.strips * p.tiles, kGsUnits) : gs_blocks(p.strips, p.groups));
}

template <typename T, bool COUPLED> hipError_t fwd_launch(const GsPlan& p, const GsArgs& a, hipStream_t s) {
    const dim3 grid(gs_grid(p));
    prof_begin(s, "gated_scan_fwd");
#define DN_GS(W, G) hipLaunchKernelGGL((gated_scan_fwd_kernel<T, COUPLED, W, G>), grid, dim3(64 * W), 0, s, a)
    if (p.chain)
        hipLaunchKernelGGL((gated_scan_fwd_chain_kernel<T, COUPLED>), grid, dim3(64 * kGsWavesC), 0, s, a);
    else if (p.waves == 1)
        DN_GS(1, 1);
    else if (p.waves == 4)
        DN_GS(4, 1);
    else if (p.waves == 16)
        DN_GS(16, 1);
    else if (p.groups == 1)
        DN_GS(8, 1);
    else if (p.groups == 2)
        DN_GS(8, 2);
    else if (p.groups == 4)
        DN_GS(8, 4);
    else
        DN_GS(8, 8);
#undef DN_GS
    prof_end(s);
    return hipGetLastError();
}
template <typename T, bool COUPLED> hipError_t bwd_launch(const GsPlan& p, const GsArgs& a, hipStream_t s) {
    const dim3 grid(gs_grid(p));
    prof_begin(s, "gated_scan_bwd");
#define DN_GS(W, G) hipLaunchKernelGGL((gated_scan_bwd_kernel<T, COUPLED, W, G>), grid, dim3(64 * W), 0, s, a)
    if (p.chain)
        hipLaunchKernelGGL((gated_scan_bwd_chain_kernel<T, COUPLED>), grid, dim3(64 * kGsWavesB), 0, s, a);
    else if (p.waves == 1)
        DN_GS(1, 1);
    else if (p.waves == 4)
        DN_GS(4, 1);
    else if (p.groups == 1)
        DN_GS(8, 1);
    else if (p.groups == 2)
        DN_GS(8, 2);
    else if (p.groups == 4)
        DN_GS(8, 4);
    else
        DN_GS(8, 8);
#undef DN_GS
    prof_end(s);
    return hipGetLastError();
}
hipError_t fwd_any(const GsProblem& pr, const GsPlan& p, const GsArgs& a, int first_tile, hipStream_t s) {
    if (p.chain) {
        const hipError_t e = clear_chain(p, a.chain, first_tile, s);
        if (e != hipSuccess) return e;
    }
    if (pr.bf16) return pr.coupled ? fwd_launch<bf16, true>(p, a, s) : fwd_launch<bf16, false>(p, a, s);
    return pr.coupled ? fwd_launch<float, true>(p, a, s) : fwd_launch<float, false>(p, a, s);
}
hipError_t bwd_any(const GsProblem& pr, const GsPlan& p, const GsArgs& a, int first_tile, hipStream_t s) {
    if (p.chain) {
        const hipError_t e = clear_chain(p, a.chain, first_tile, s);
        if (e != hipSuccess) return e;
    }
    if (pr.bf16) return pr.coupled ? bwd_launch<bf16, true>(p, a, s) : bwd_launch<bf16, false>(p, a, s);
    return pr.coupled ? bwd_launch<float, true>(p, a, s) : bwd_launch<float, false>(p, a, s);
}

}  // namespace

hipError_t launch_gated_scan_fwd(const GsProblem& pr, const GsFwd& f, char* ws, hipStream_t s) {
    if (pr.B == 0 || pr.H == 0) return hipSuccess;
    const GsPlan p = gs_plan(pr, false);
    GsArgs a = gs_args(pr, p, f.x, f.g, f.lens, ws);
    a.first = f.h0;
    a.out = f.o;
    a.last = f.hT;
    a.states = f.states;
    return fwd_any(pr, p, a, f.first_tile, s);
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
        const hipError_t e = fwd_any(pr, p, a, 0, s);
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
    return bwd_any(pr, p, a, f.first_tile, s);
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
