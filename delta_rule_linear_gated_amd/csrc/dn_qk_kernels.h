// dn_qk_kernels.h -- norms of queries and keys for each head and their rotation by position,
// in one pass over the rows, and its backward pass:
//     r = (share |x|^2 + eps)^{-1/2},   n = r x * w,   y = R(theta_t) n,
//     u = R(-theta_t) dy,   e = w * u,   dx = r (e - share r^2 <x, e> x),   dw = sum r x * u.
//
// A row of d elements takes d / 8 lanes of 8 elements: two pieces of four, so that both
// members of every rotated pair lie in one lane (halves: elements 4p and rot / 2 + 4p on; else,
// and in the part that is not rotated, 8p on) and only the row's sum crosses lanes.  A lane
// keeps its token (its angles: fp64, reduced to an eighth turn, then short series) over the
// heads of a group.  The bytes of the rows are what bounds it, read and written once, four rows of
// a lane in flight (backward: two of each tensor).  At 32 + 32 heads of 128, 32768 steps, bf16: l2
// 211 us (5.1 TB/s), rms with halves rotated 220, rotation alone 215, backward of l2 304 (5.3 TB/s),
// of rms with rotation and weights 323; a large copy runs at 5.1 to 5.2.
#pragma once

#include "dn_device.h"
#include "dn_qk.h"

namespace dn {

constexpr int kQkThreads = 256;
constexpr int kQkHeads = 4;   // rows of a lane in flight

__device__ __forceinline__ f32x4 qk_load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ uint2 qk_load4(const bf16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void qk_open(const f32x4& v, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
}
__device__ __forceinline__ void qk_open(const uint2& v, float* x) {
    x[0] = __builtin_bit_cast(float, v.x << 16);
    x[1] = __builtin_bit_cast(float, v.x & 0xffff0000u);
    x[2] = __builtin_bit_cast(float, v.y << 16);
    x[3] = __builtin_bit_cast(float, v.y & 0xffff0000u);
}
// Both pieces of a lane's row: one after the other in memory unless halves are rotated.
template <typename T> struct QkRow;
template <> struct QkRow<float> {
    f32x4 a, b;
    template <bool APART> __device__ __forceinline__ void load(const float* p, int at, int bt) {
        a = qk_load4(p + at);
        b = qk_load4(p + bt);
    }
    __device__ __forceinline__ void open(float (&x)[8]) const { qk_open(a, x), qk_open(b, x + 4); }
    template <bool APART> static __device__ __forceinline__ void store(float* p, int at, int bt, const float (&x)[8]) {
        *reinterpret_cast<f32x4*>(p + at) = f32x4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4*>(p + bt) = f32x4{x[4], x[5], x[6], x[7]};
    }
};
template <> struct QkRow<bf16> {
    uint2 a, b;
    template <bool APART> __device__ __forceinline__ void load(const bf16* p, int at, int bt) {
        if (APART) {
            a = qk_load4(p + at);
            b = qk_load4(p + bt);
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(p + at);
            a = make_uint2(v.x, v.y);
            b = make_uint2(v.z, v.w);
        }
    }
    __device__ __forceinline__ void open(float (&x)[8]) const { qk_open(a, x), qk_open(b, x + 4); }
    template <bool APART> static __device__ __forceinline__ void store(bf16* p, int at, int bt, const float (&x)[8]) {
        typedef __attribute__((ext_vector_type(4))) __bf16 b4;
        const b4 u{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]}, v{(bf16)x[4], (bf16)x[5], (bf16)x[6], (bf16)x[7]};
        if (APART) {
            *reinterpret_cast<b4*>(p + at) = u;
            *reinterpret_cast<b4*>(p + bt) = v;
        } else {
            const uint2 lo = __builtin_bit_cast(uint2, u), hi = __builtin_bit_cast(uint2, v);
            *reinterpret_cast<uint4*>(p + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
};

// cos and sin of pos * freq times the amplitude.  The angle is reduced in 64 bits to at most
// an eighth of a turn around a multiple of a quarter (both parts of pi / 2: the reduced angle
// of a far position keeps what the product has), where the series to the ninth and tenth
// power leave less than half a step of fp32.
__device__ __forceinline__ void qk_angle(double pos, double freq, float amp, float& c, float& s) {
    const double t = pos * freq, k = rint(t * 0.63661977236758134308);
    double r = fma(k, -1.57079632679489655800, t);
    r = fma(k, -6.12323399573676603587e-17, r);
    const float x = (float)r, z = x * x;
    float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    sn = fmaf(sn, z, 1.f / 120.f);
    sn = fmaf(sn, z, -1.f / 6.f);
    sn = fmaf(sn * z, x, x);
    float cs = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
    cs = fmaf(cs, z, -1.f / 720.f);
    cs = fmaf(cs, z, 1.f / 24.f);
    cs = fmaf(cs, z, -0.5f);
    cs = fmaf(cs, z, 1.f);
    const int quarter = (int)((k * 0.25 - floor(k * 0.25)) * 4.0);
    const float u = quarter & 1 ? sn : cs, v = quarter & 1 ? cs : sn;
    c = (quarter + 1) & 2 ? -u * amp : u * amp;
    s = quarter & 2 ? -v * amp : v * amp;
}

// The lane's pairs rotated in place: (i, i + 4) for halves, (2i, 2i + 1) for neighbours.
template <int TURN> __device__ __forceinline__ void qk_turn(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = TURN == kTurnHalves ? i : 2 * i, n = TURN == kTurnHalves ? i + 4 : 2 * i + 1;
        const float u = x[m], v = x[n];
        x[m] = fmaf(u, c[i], -v * s[i]);
        x[n] = fmaf(v, c[i], u * s[i]);
    }
}

template <int D> __device__ __forceinline__ float qk_row_sum(float x) { return group_sum<D / 8>(x); }

// Where a lane works: its token, its elements, its angles.
struct QkPlace {
    int b, t, at, bt;
    bool there, live, turned;   // a token of the batch, before its sequence's end, in the rotated part
};
template <int D, int TURN> __device__ __forceinline__ void qk_place(const QkArgs& a, int m, int p, QkPlace& k) {
    k.there = m < a.B * a.T;
    k.b = k.there ? m / a.T : 0;
    k.t = k.there ? m - k.b * a.T : 0;
    k.live = k.there && (!a.lens || k.t < a.lens[k.b]);
    k.turned = TURN != kTurnNone && 8 * p < a.rot;
    k.at = TURN == kTurnHalves && k.turned ? 4 * p : 8 * p;
    k.bt = TURN == kTurnHalves && k.turned ? a.rot / 2 + 4 * p : 8 * p + 4;
}
__device__ __forceinline__ void qk_angles(const QkArgs& a, const QkPlace& k, int p, float sign, float (&c)[4], float (&s)[4]) {
    if (!k.turned || !k.live) return;
    const double pos = a.pos_kind == 0 ? (double)k.t
                       : a.pos_kind == 1 ? (double)a.pos[k.b] + k.t
                                         : (double)a.pos[(long)k.b * a.T + k.t];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        qk_angle(pos, a.freqs[4 * p + i], a.amplitude, c[i], s[i]);
        s[i] *= sign;
    }
}

// The head group of a workgroup: side, first head, heads.
__device__ __forceinline__ void qk_group(const QkArgs& a, int group, int& side, int& h0, int& n) {
    side = group >= a.groups[0];
    if (side) group -= a.groups[0];
    h0 = group * a.per;
    n = min(a.per, a.side[side].heads - h0);
}

// The token tile of a workgroup in a round of a.tiles.  Shifted from round to round: at equal steps
// a workgroup could find the same steps of every sequence, and the ends of a padded batch leave
// half of the workgroups without work.
__device__ __forceinline__ long qk_tile(const QkArgs& a, int round) {
    const int shift = (int)((long)a.tiles * 5 / 8);
    return round * (long)a.tiles + (blockIdx.x % a.tiles + round * (long)shift) % a.tiles;
}

// Grid: workgroups that walk the token tiles of their head group.
template <typename T, int D, int TURN, bool NORM> __global__ __launch_bounds__(kQkThreads) void qk_fwd_kernel(QkArgs a) {
    constexpr int LANES = D / 8, TOKENS = kQkThreads / LANES;
    constexpr bool APART = TURN == kTurnHalves;
    const int p = threadIdx.x % LANES;
    int sd, h0, nh;
    qk_group(a, blockIdx.x / a.tiles, sd, h0, nh);
    const QkSide& S = a.side[sd];
    QkPlace k;
    qk_place<D, TURN>(a, 0, p, k);   // the lane's elements are the same for every token
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = NORM && S.w ? S.w[i < 4 ? k.at + i : k.bt + i - 4] : 1.f;
    const long tokens = (long)a.B * a.T;
    for (int round = 0; round * (long)a.tiles * TOKENS < tokens; ++round) {
        const long m0 = qk_tile(a, round) * TOKENS;
        if (m0 >= tokens) continue;
        qk_place<D, TURN>(a, (int)min(m0 + threadIdx.x / LANES, tokens), p, k);
        float c[4], s[4];
        const T* x = static_cast<const T*>(S.x) + k.b * S.xs[0] + h0 * S.xs[1] + k.t * S.xs[2];
        T* y = static_cast<T*>(S.out) + k.b * S.os[0] + h0 * S.os[1] + k.t * S.os[2];
        QkRow<T> rows[kQkHeads];
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < kQkHeads; ++i)
                if (k.live && h + i < nh) rows[i].template load<APART>(x + (h + i) * S.xs[1], k.at, k.bt);
        };
        fetch(0);
        if (TURN != kTurnNone) qk_angles(a, k, p, a.back ? -1.f : 1.f, c, s);
        for (int h = 0; h < nh; h += kQkHeads) {
            if (h) fetch(h);
#pragma unroll
            for (int i = 0; i < kQkHeads; ++i) {
                if (h + i >= nh) break;
                float v[8] = {};
                if (k.live) rows[i].open(v);
                if (NORM) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
                    const float r = rsqrtf(fmaf(qk_row_sum<D>(sum), a.share, a.eps));
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] * r * w[j];
                }
                if (TURN != kTurnNone && k.turned) qk_turn<TURN>(v, c, s);
                if (!k.live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.f;
                }
                if (k.there) QkRow<T>::template store<APART>(y + (h + i) * S.os[1], k.at, k.bt, v);
            }
        }
    }
}

// Backward of a norm (with or without a rotation).  Grid: workgroups that walk the token
// tiles of their head group in steps of a.tiles; dw of a workgroup's rows goes to its entry
// of parts.
template <typename T, int D, int TURN, bool DW> __global__ __launch_bounds__(kQkThreads) void qk_bwd_kernel(QkArgs a) {
    constexpr int LANES = D / 8, TOKENS = kQkThreads / LANES;
    constexpr bool APART = TURN == kTurnHalves;
    constexpr int ROWS = kQkHeads / 2;   // two tensors: as many bytes in flight
    const int p = threadIdx.x % LANES;
    int sd, h0, nh;
    qk_group(a, blockIdx.x / a.tiles, sd, h0, nh);
    const QkSide& S = a.side[sd];
    QkPlace k;
    qk_place<D, TURN>(a, 0, p, k);   // the lane's elements are the same for every token
    float w[8], dw[8] = {}, over[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = S.w ? S.w[i < 4 ? k.at + i : k.bt + i - 4] : 1.f;
    const long ystep = (long)a.T * D, tokens = (long)a.B * a.T;
    for (int round = 0; round * (long)a.tiles * TOKENS < tokens; ++round) {
        const long m0 = qk_tile(a, round) * TOKENS;
        if (m0 >= tokens) continue;
        qk_place<D, TURN>(a, (int)min(m0 + threadIdx.x / LANES, tokens), p, k);
        float c[4], s[4];
        const T* x = static_cast<const T*>(S.x) + k.b * S.xs[0] + h0 * S.xs[1] + k.t * S.xs[2];
        const T* dy = static_cast<const T*>(S.dy) + (((long)k.b * S.heads + h0) * a.T + k.t) * D;
        T* dx = static_cast<T*>(S.out) + k.b * S.os[0] + h0 * S.os[1] + k.t * S.os[2];
        QkRow<T> rx[ROWS], ry[ROWS];
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                if (k.live && h + i < nh) {
                    rx[i].template load<APART>(x + (h + i) * S.xs[1], k.at, k.bt);
                    ry[i].template load<APART>(dy + (h + i) * ystep, k.at, k.bt);
                }
        };
        float sum[8] = {};   // of the token's heads
        fetch(0);
        if (TURN != kTurnNone) qk_angles(a, k, p, -1.f, c, s);
        for (int h = 0; h < nh; h += ROWS) {
            if (h) fetch(h);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (h + i >= nh) break;
                float v[8] = {}, u[8] = {}, sq = 0.f, xe = 0.f;
                if (k.live) rx[i].open(v), ry[i].open(u);
                if (TURN != kTurnNone && k.turned) qk_turn<TURN>(u, c, s);
#pragma unroll
                for (int j = 0; j < 8; ++j) sq = fmaf(v[j], v[j], sq);
                const float r = rsqrtf(fmaf(qk_row_sum<D>(sq), a.share, a.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] *= r;   // the unit row
                    if (DW && k.live) sum[j] = fmaf(v[j], u[j], sum[j]);
                    u[j] *= w[j];
                    xe = fmaf(v[j], u[j], xe);
                }
                xe = qk_row_sum<D>(xe) * a.share;
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = k.live ? r * fmaf(-xe, v[j], u[j]) : 0.f;
                if (k.there) QkRow<T>::template store<APART>(dx + (h + i) * S.os[1], k.at, k.bt, u);
            }
        }
        if (!DW) continue;
        // The tokens of a lane may be many thousands: what each addition rounds off is added up by itself
        // (over), so that the error does not grow with them: 2^24 equal rows, 8 heads, 255 half steps of
        // fp32 -> 16.  Time: none where rows are many, half a microsecond and up to 1 of 20 with few (one head
        // of 16, 39 sequences of 10220 steps).
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float to = dw[j] + sum[j];
            over[j] += (to - dw[j]) - sum[j];
            dw[j] = to;
        }
    }
    if (!DW) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = fabsf(over[j]) < __builtin_inff() ? dw[j] - over[j] : dw[j];   // not of an infinite sum
    // over the tokens of the workgroup: lanes of the same elements, then the waves
    __shared__ float part[kQkThreads / 64][D];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int step = LANES; step < 64; step *= 2) dw[j] += __shfl_xor(dw[j], step);
        if (lane_id() < LANES) part[wave_id()][j < 4 ? k.at + j : k.bt + j - 4] = dw[j];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += kQkThreads) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < kQkThreads / 64; ++v) sum += part[v][j];
        a.parts[(long)blockIdx.x * D + j] = sum;
    }
}

template <typename T, int D> hipError_t qk_fwd_width(const QkArgs& a, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(kQkThreads);
#define DN_QK(TURN, NORM) hipLaunchKernelGGL((qk_fwd_kernel<T, D, TURN, NORM>), grid, block, 0, s, a)
    if (a.norm) {
        if (a.turn == kTurnNone)
            DN_QK(kTurnNone, true);
        else if (a.turn == kTurnHalves)
            DN_QK(kTurnHalves, true);
        else
            DN_QK(kTurnNeighbours, true);
    } else {
        if (a.turn == kTurnHalves)
            DN_QK(kTurnHalves, false);
        else
            DN_QK(kTurnNeighbours, false);
    }
#undef DN_QK
    return hipGetLastError();
}
template <typename T, int D> hipError_t qk_bwd_width(const QkArgs& a, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(kQkThreads);
    const bool dw = a.side[0].dw || a.side[1].dw;
#define DN_QK(TURN)                                                                      \
    if (dw)                                                                              \
        hipLaunchKernelGGL((qk_bwd_kernel<T, D, TURN, true>), grid, block, 0, s, a);     \
    else                                                                                 \
        hipLaunchKernelGGL((qk_bwd_kernel<T, D, TURN, false>), grid, block, 0, s, a)
    if (a.turn == kTurnNone) {
        DN_QK(kTurnNone);
    } else if (a.turn == kTurnHalves) {
        DN_QK(kTurnHalves);
    } else {
        DN_QK(kTurnNeighbours);
    }
#undef DN_QK
    return hipGetLastError();
}
template <typename T> hipError_t qk_fwd_type(const QkArgs& a, unsigned blocks, hipStream_t s) {
    switch (a.d) {
        case 16: return qk_fwd_width<T, 16>(a, blocks, s);
        case 32: return qk_fwd_width<T, 32>(a, blocks, s);
        case 64: return qk_fwd_width<T, 64>(a, blocks, s);
        case 128: return qk_fwd_width<T, 128>(a, blocks, s);
        default: return hipErrorInvalidValue;
    }
}
template <typename T> hipError_t qk_bwd_type(const QkArgs& a, unsigned blocks, hipStream_t s) {
    switch (a.d) {
        case 16: return qk_bwd_width<T, 16>(a, blocks, s);
        case 32: return qk_bwd_width<T, 32>(a, blocks, s);
        case 64: return qk_bwd_width<T, 64>(a, blocks, s);
        case 128: return qk_bwd_width<T, 128>(a, blocks, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace dn
