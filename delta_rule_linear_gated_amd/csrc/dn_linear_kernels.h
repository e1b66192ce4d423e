// dn_linear_kernels.h -- the chunk kernel of linear attention with a decay per
// head (see LinOp in dn_linear.h).
//
// A workgroup takes one (b, h), one block of VB channels of z, and a run of
// chunks of 64 steps in order.  The state block S [VB][KD] stays in fp32
// accumulators for the whole run, so HBM sees x, y, z once and out once.  With
// G the running log-decay of the chunk (base 2, summed in 64 bits and kept as two
// floats, so that differences of close steps stay exact far down the decay):
//     out^T = (S x^T) e^{G_i}  +  z^T P^T,   P^T = (y x^T) e^{G_i - G_j}, j <= i
//     S^T   = e^{G_63} S^T + y^T (z e^{G_63 - G_j})
// Every product is formed transposed so that its accumulator is the next one's
// operand or a row piece in memory: P^T stays in registers (a lane's four
// accumulator rows are four consecutive K slots of the product with z), out^T
// gives a lane 16-byte pieces of one step's channels, S^T four consecutive channels
// of y.  Four waves form the outputs, 16 steps each; four more the state, so
// that the two halves of a chunk's work, which only share the tiles, run side by side.
//
// Rounding (bf16 I/O): P and S enter the products that form an output as two bf16 parts
// each (what they leave is at most 2^-16 of a term, wherever in the run the chunk is), so
// that an output's error is its own rounding.  With S as one part, rounded like the
// outputs, their error was 1.1 to 1.4 roundings and differed with the split of the steps
// (8 x 16 heads, 4096 ragged steps: 143 us against 163; 32 heads, 32768 steps, train step:
// 1315 against 1525).  The state itself is held to fp32: its operand z e^{..} enters as
// three bf16 parts (24 bits), since a state (hT, dh0) is an fp32 output.  Where the gate's
// gradient is wanted, an fp32 sum of differences of r . out, P and S enter in three
// parts too, and P's diagonal, which is no part of that gradient, is applied apart from
// the others.
// fp32 I/O: every product on fp32 matrix-core steps.
//
// Measured (bf16, d = 128, one workgroup on a compute unit; kernel traces of whole, warm runs).
// Forward, 8 x 16 heads, 4096 steps: 152 us for 0.55 GB, 3.6 TB/s where a copy reaches 5.2;
// its matrix (36 % busy) and LDS (56 %) work overlap in part only.  32 heads, 32768 steps in
// 8 segments: 137 us for their states, 8 to join them, 287 for the outputs (3.8 TB/s); backward in
// one run, 1048 us.  With the gate's gradient, 8 x 16 heads, 4096 steps, two evaluations: 512 us
// for 1.4 GB; LDS 46 %, matrix 27 % busy.  Blocks of 64 channels of z: of 32, x y^T is formed
// twice as often (219 us where these took 150).
#pragma once

#include <type_traits>

#include "dn_device.h"
#include "dn_linear.h"
#include "dn_split.h"

namespace dn {

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

template <typename T> struct LinT;
template <> struct LinT<bf16> {
    typedef bf16x8 Frag;                                // 8 K slots of one row
    static constexpr int E = 8, JS = 32;                // elements of a fragment; K of one transposed step
    __device__ __forceinline__ static f32x4 mma(Frag a, Frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    // K over rows row0 + {4 g + i, 16 + 4 g + i}; operand row m is column col4(m / 4) + m % 4
    // (col: the piece of this lane, col4(lane % 4))
    __device__ __forceinline__ static Frag load_t(const bf16* p, int ld, int row0, int col) {
        const int l = lane_id(), i = l & 15;
        const bf16* a = p + (row0 + 4 * (l >> 4) + (i >> 2)) * ld + col;
        const i16x4 v[2] = {tr16_b64(a), tr16_b64(a + 16 * ld)};
        return *reinterpret_cast<const bf16x8*>(v);
    }
};
template <> struct LinT<float> {
    typedef f32x4 Frag;
    static constexpr int E = 4, JS = 16;
    __device__ __forceinline__ static f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
    // K over rows row0 + 4 g + i; col: this lane's own column
    __device__ __forceinline__ static Frag load_t(const float* p, int ld, int row0, int col) {
        const float* a = p + (row0 + 4 * (lane_id() >> 4)) * ld + col;
        return Frag{a[0], a[ld], a[2 * ld], a[3 * ld]};
    }
};

// Buffer accesses: loads past the range give zero, stores past it do nothing, so that
// rows past a sequence's end need neither branches (behind which the compiler would
// wait for every access in flight, the outputs' stores among them: 1.8 times the time of
// a chunk) nor selects.  The base is uniform; kNowhere is past every range.
typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2;
constexpr int kNowhere = 0x7ffffff0;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lin_range(const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes > 0 ? bytes : 0, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, int at) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
}

// LDS rows of y and z are padded for the transposed reads, which take four rows of 32
// bytes at once (bf16: rows 8 dwords apart modulo 64, or a permutation of that).
template <typename T, int KD, int NV, int MODE> struct LinLds {
    static constexpr bool DG = MODE == kLinDots;
    static constexpr int VB = 16 * NV, E = 16 / sizeof(T), PAD = sizeof(T) == 2 ? 2 * E : E;
    static constexpr int LY = KD + PAD, LZ = VB + PAD, LS = KD + E;
    static constexpr int NS = MODE == kLinState ? 0 : sizeof(T) == 2 ? DG ? 3 : 2 : 1;   // parts of the state operand
    T y[kLinC * LY];
    T z[kLinC * LZ];
    // The state operand.  bf16: double, so that the waves of the state, which are done before those
    // of the outputs, write the next chunk's at once (one buffer would leave room for a second
    // workgroup on a unit at d = 128, but took 180 us where two take 163, 8 x 16 heads, 4096 ragged
    // steps); with fp32 rows it is the state that the others wait for.
    static constexpr bool TWO = sizeof(T) == 2 && MODE != kLinState;
    T s[TWO ? 2 * NS : NS > 0 ? NS : 1][NS > 0 ? VB * LS : 1];
    // R: G from the first step of the row's 16 (two floats); e^{G_63 - G};
    // e^{G_16w - G_j} of the rows j before 16 w, w = 1, 2, 3; e^{G_16w}; the chunk's factor
    float hi[kLinC], lo[kLinC], ew[kLinC], tab[3][kLinC], eref[4], etot;
    static constexpr int HV = lin_halves(MODE, sizeof(T) == 2, NV);
    float dot[2][HV][HV > 1 ? kLinC : 1];
};

// Gate that the state takes when step t is entered: the step's own, or with rev that of
// the step after it; none past the length.  The load is free of branches (addresses
// clamped), so that nothing waits for it before lin_log2 uses it.
__device__ __forceinline__ float lin_gate(const LinArgs& a, const float* g, int n, int t, int rev) {
    const int at = rev ? t + 1 : t;
    return a.gate == kLinNone ? 0.f : g[a.gate == kLinScalar ? min(at, n - 1) : 0];
}
// Its logarithm to base 2.  Below -1000 a factor is zero in fp32 whatever the rest, so
// that -inf (a reset) gives no inf - inf; NaN stays.
__device__ __forceinline__ double lin_log2(float g, int n, int t, int rev) {
    if ((rev ? t + 1 : t) >= n) return 0.0;
    return (double)(g < -1000.f ? -1000.f : g) * 1.4426950408889634;
}

// Sums in 64 bits over the lanes of a wave up to each, and the value of one lane, on the
// vector ALU alone (a scan by LDS permutes took a quarter of a chunk's time in the wave
// that makes it): DPP row_shr 1, 2, 4, 8, then row_bcast 15 and 31 into the rows behind.
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_add(double x) {
    const uint2 u = __builtin_bit_cast(uint2, x);
    const uint2 v = make_uint2((unsigned)__builtin_amdgcn_update_dpp(0, (int)u.x, CTRL, ROWS, 0xF, false),
                               (unsigned)__builtin_amdgcn_update_dpp(0, (int)u.y, CTRL, ROWS, 0xF, false));
    return x + __builtin_bit_cast(double, v);
}
__device__ __forceinline__ double wave_scan(double x) {
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    return dpp_add<0x143, 0xC>(x);
}
__device__ __forceinline__ double of_lane(double x, int l) {
    const uint2 u = __builtin_bit_cast(uint2, x);
    return __builtin_bit_cast(double, make_uint2((unsigned)__builtin_amdgcn_readlane((int)u.x, l),
                                                 (unsigned)__builtin_amdgcn_readlane((int)u.y, l)));
}

template <typename T, int KD, int NV, int MODE>
__global__ __launch_bounds__(lin_threads(MODE, sizeof(T) == 2, NV), lin_waves(MODE, sizeof(T) == 2, KD, NV)) void lin_kernel(LinArgs a) {
    constexpr bool OUT = MODE != kLinState, DG = MODE == kLinDots;
    constexpr int TH = lin_threads(MODE, sizeof(T) == 2, NV), HV = lin_halves(MODE, sizeof(T) == 2, NV);
    using X = LinT<T>;
    using Frag = typename X::Frag;
    using L = LinLds<T, KD, NV, MODE>;
    constexpr int E = X::E, JS = X::JS, VB = 16 * NV, LY = L::LY, LZ = L::LZ, LS = L::LS, NS = L::NS;
    constexpr int NVW = NV / HV;                             // output tiles of a wave
    constexpr int XF = KD / (4 * E);                         // fragments of an x row
    constexpr int WV = 4 / NV;                               // waves that share a state tile column
    constexpr int CT = KD / 16 / WV > 0 ? KD / 16 / WV : 1;  // state tiles of a wave
    constexpr int PY = KD / E, NY = (kLinC * PY + TH - 1) / TH;   // 16-byte pieces
    constexpr int PZ = VB / E, NZ = (kLinC * PZ + TH - 1) / TH;
    __shared__ __align__(16) L s;
    // z channel of accumulator element i of lane group q in output tile `tile`: a lane's
    // elements of TP tiles are 16 bytes of a row, and the four groups' follow each other
    constexpr int TP = lin_pair(sizeof(T) == 2, NV);
    auto out_col = [](int tile, int q, int i) { return 16 * TP * (tile / TP) + 4 * TP * q + 4 * (tile % TP) + i; };

    // Workgroups go to the 8 XCDs in turn: the blocks and evaluations of one (b, h) and
    // segment, which read the same rows, get ids equal mod 8 (one L2).
    const int sub = a.nops * a.nblk;
    const int slot = blockIdx.x / kXcds;
    const int unit = (slot / sub) * kXcds + blockIdx.x % kXcds;
    if (unit >= a.BH * a.nseg) return;
    const int oi = (slot % sub) / a.nblk, blk = slot % a.nblk;
    const int bh = unit / a.nseg, seg = unit % a.nseg;
    const LinOp& op = a.op[oi];
    const int rev = op.rev;
    if (!OUT && (rev ? seg == 0 : seg == a.nseg - 1)) return;   // nothing starts from its end

    // waves 0 .. 4 HV - 1 form the outputs (16 steps each, HV shares of the channels), the
    // others the state
    const int tid = threadIdx.x, l = lane_id(), g = l >> 4, m = l & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;   // uniform: branches on it are scalar
    const int h = bh % a.H, n = __builtin_amdgcn_readfirstlane(lin_len(a.lens, bh / a.H, a.T));
    const int c0 = seg * a.seg_len, c1 = min(a.NT, c0 + a.seg_len);
    const int cv = min(c1, (n + kLinC - 1) / kLinC);   // chunks past it hold no step
    const long rows = (long)bh * a.T;
    const T* xp = static_cast<const T*>(op.x) + rows * a.kd;
    const T* yp = static_cast<const T*>(op.y) + rows * a.kd;
    const T* zp = static_cast<const T*>(op.z) + rows * a.nd + blk * VB;
    const int vt = w % NV, ct0 = (w / NV) * CT;        // this wave's state tiles
    const bool owns = ct0 * 16 < KD;
    const int vrow = blk * VB + 16 * vt + m;           // the state row of this lane
    const float* gp = a.gate == kLinNone ? nullptr : a.gate == kLinHead ? a.g + h : a.g + rows;

    float* snap = op.snap ? op.snap + bh * op.snap_bh : nullptr;
    const long se = (long)a.kd * a.nd;                        // floats of a kept state
    const int ent0 = rev ? (c1 - 1) / a.snap : c0 / a.snap;   // the segment's first entry
    const int step = rev ? -1 : 1, first = rev ? cv - 1 : c0, count = cv - c0;
    const int trow = 16 * w + m;                              // an output lane's step within the chunk
    auto time_of = [&](int c, int row) { return c * kLinC + (rev ? kLinC - 1 - row : row); };

    // The run of one wave of the outputs (O) or of the state: the same barriers in both, and
    // registers for one of them only.
    auto run = [&](auto outs) {
        constexpr bool O = decltype(outs)::value;
        const int half = O ? wave >> 2 : 0, tile0 = half * NVW;   // this wave's output tiles
        // ---- tiles of a chunk: 16-byte pieces, places in bytes from the chunk's first row
        u32x4 yr[NY], zr[NZ];
        Frag xn[O ? XF : 1], x[O ? XF : 1];
        T rn[O && DG ? 4 * NVW : 1], r[O && DG ? 4 * NVW : 1];
        auto row_at = [&](int row, int width) { return (rev ? kLinC - 1 - row : row) * width * (int)sizeof(T); };
        int yo[NY], zo[NZ];
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int id = tid + TH * i, col = (id % PY) * E;
            yo[i] = col < a.kd && id / PY < kLinC ? row_at(id / PY, a.kd) + col * (int)sizeof(T) : kNowhere;
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
            const int id = tid + TH * i;
            zo[i] = id / PZ < kLinC ? row_at(id / PZ, a.nd) + (id % PZ) * 16 : kNowhere;
        }
        const int xo = row_at(trow, a.kd) + 16 * g;
        auto load = [&](int c) {
            const int row0 = c * kLinC, live = min(n - row0, kLinC);
            const auto yb = lin_range(yp + (long)row0 * a.kd, live * a.kd * (int)sizeof(T));
            const auto zb = lin_range(zp + (long)row0 * a.nd, (live * a.nd - blk * VB) * (int)sizeof(T));
#pragma unroll
            for (int i = 0; i < NY; ++i) yr[i] = load16(yb, yo[i]);
#pragma unroll
            for (int i = 0; i < NZ; ++i) zr[i] = load16(zb, zo[i]);
            if constexpr (O) {
                const auto xb = lin_range(xp + (long)row0 * a.kd, live * a.kd * (int)sizeof(T));
#pragma unroll
                for (int f = 0; f < XF; ++f)
                    xn[f] = __builtin_bit_cast(
                        Frag, load16(xb, KD > 32 || 4 * E * f + E * g < a.kd ? xo + 64 * f : kNowhere));
            }
            if constexpr (O && DG) {   // rows of the other factor of the gate's gradient, the lane's output channels
                const auto rb = lin_range(static_cast<const T*>(op.r) + (rows + row0) * a.nd + blk * VB,
                                          (min(n - row0, kLinC) * a.nd - blk * VB) * (int)sizeof(T));
#pragma unroll
                for (int i = 0; i < NVW; i += TP) {
                    const int at = row_at(trow, a.nd) + out_col(tile0 + i, g, 0) * (int)sizeof(T);
                    if constexpr (TP * 4 * sizeof(T) == 16) {
                        const Frag v = __builtin_bit_cast(Frag, load16(rb, at));
#pragma unroll
                        for (int e = 0; e < E; ++e) rn[4 * i + e] = v[e];
                    } else {
                        typedef typename Vec4<T>::type V4;
                        const V4 v = __builtin_bit_cast(V4, __builtin_amdgcn_raw_buffer_load_b64(rb, at, 0, 0));
#pragma unroll
                        for (int e = 0; e < 4; ++e) rn[4 * i + e] = v[e];
                    }
                }
            }
        };
        auto put_tiles = [&]() {
#pragma unroll
            for (int i = 0; i < NY; ++i) {
                const int id = tid + TH * i;
                if (kLinC * PY % TH == 0 || id / PY < kLinC)
                    *reinterpret_cast<u32x4*>(&s.y[(id / PY) * LY + (id % PY) * E]) = yr[i];
            }
#pragma unroll
            for (int i = 0; i < NZ; ++i) {
                const int id = tid + TH * i;
                if (kLinC * PZ % TH == 0 || id / PZ < kLinC)
                    *reinterpret_cast<u32x4*>(&s.z[(id / PZ) * LZ + (id % PZ) * E]) = zr[i];
            }
            if constexpr (O) {
#pragma unroll
                for (int f = 0; f < XF; ++f) x[f] = xn[f];
            }
            if constexpr (O && DG) {
#pragma unroll
                for (int e = 0; e < 4 * NVW; ++e) r[e] = rn[e];
            }
        };
        // ---- running log-decay of a chunk: lane = row, sums in 64 bits.  One wave forms it
        // (of the outputs' the one with the fewest pairs under the diagonal) and holds it
        // until the chunk before is done.
        const bool gates = wave == 0;
        double dec = 0.0;                                  // of the run so far
        float ghi = 0.f, glo = 0.f, gew = 0.f, gtab[4] = {}, getot = 0.f, geref = 0.f;
        auto form_gates = [&](double x2) {
            x2 = wave_scan(x2);
            const double tot = of_lane(x2, 63), at[4] = {of_lane(x2, 0), of_lane(x2, 16), of_lane(x2, 32), of_lane(x2, 48)};
            const double own = g < 2 ? (g == 0 ? at[0] : at[1]) : (g == 2 ? at[2] : at[3]);   // of the row's block
            ghi = (float)(x2 - own), glo = (float)(x2 - own - (double)ghi);
            gew = exp2_hw((float)(tot - x2));
            getot = exp2_hw((float)tot);
            geref = exp2_hw((float)own);
            if constexpr (OUT) {
#pragma unroll
                for (int u = 1; u < 4; ++u) gtab[u] = exp2_hw((float)(at[u] - x2));
            }
            dec += tot;
        };
        auto put_gates = [&]() {
            s.ew[l] = gew;
            if (l == 0) s.etot = getot;
            if constexpr (OUT) {
                s.hi[l] = ghi, s.lo[l] = glo;
                if ((l & 15) == 0) s.eref[l >> 4] = geref;
#pragma unroll
                for (int u = 1; u < 4; ++u) s.tab[u - 1][l] = gtab[u];
            }
        };
        auto put_dot = [&](int which, int c, int at, float d) {
            const auto db = lin_range(op.dots + (((long)which * a.nblk + blk) * a.BH + bh) * a.T + c * kLinC,
                                      min(n - c * kLinC, kLinC) * 4);
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, d), db, at, 0, 0);
        };
        auto rdot = [&](const auto& acc, const auto& r) {   // over the lane's channels
            float d = 0.f;
#pragma unroll
            for (int i = 0; i < NVW; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) d += acc[i][e] * to_f(r[4 * i + e]);
            return d;
        };
        // ---- state block: element pieces of this lane in global memory and in LDS
        f32x4 S[O ? 1 : CT];
        auto each_piece = [&](auto f) {                    // f(tile, offset of its four elements)
            if (!owns) return;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int k0 = 16 * (ct0 + ct) + 4 * g;
                if (k0 < a.kd) f(ct, (long)vrow * op.sn + (long)k0 * op.sk);
            }
        };
        auto load_state = [&](const float* base) {
            each_piece([&](int ct, long at) {
                if (op.sk == 1) {
                    S[ct] = *reinterpret_cast<const f32x4*>(base + at);
                } else {
                    const long d = op.sk;
                    S[ct] = f32x4{base[at], base[at + d], base[at + 2 * d], base[at + 3 * d]};
                }
            });
        };
        auto store_state = [&](float* base, float f) {
            each_piece([&](int ct, long at) {
                const f32x4 v = S[ct] * f;
                if (op.sk == 1) {
                    *reinterpret_cast<f32x4*>(base + at) = v;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) base[at + (long)i * op.sk] = v[i];
                }
            });
        };
        auto put_state = [&](auto parts, int buf) {
            constexpr int N = decltype(parts)::value;
            if (!owns) return;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int at = buf * NS * VB * LS + (16 * vt + m) * LS + 16 * (ct0 + ct) + 4 * g;
                if constexpr (N == 1) {
                    st4<T>(&s.s[0][at], S[ct]);
                } else {
                    float v0 = S[ct][0], v1 = S[ct][1], v2 = S[ct][2], v3 = S[ct][3];
#pragma unroll
                    for (int p = 0; p < N; ++p) {
                        const u32x2 v = {take_bf16(v0, v1), take_bf16(v2, v3)};
                        *reinterpret_cast<u32x2*>(&s.s[p][at]) = v;
                    }
                }
            }
        };
        if constexpr (!O) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[ct] = zero4();
            if (OUT && a.nseg > 1)
                load_state(snap + ent0 * se);
            else if (OUT && op.init)
                load_state(op.init + bh * se);
        }

        if (count > 0) {
            const float g0 = lin_gate(a, gp, n, time_of(first, l), rev);
            load(first);
            if (gates) {
                form_gates(lin_log2(g0, n, time_of(first, l), rev));
                put_gates();
            }
            put_tiles();
            if constexpr (OUT && !O) put_state(std::integral_constant<int, NS>{}, 0);
        }
        auto chunk = [&](int ci) {
            const int c = first + step * ci;
            const int next = ci + 1 < count ? c + step : c;   // after the last chunk: it again, unused
            const int buf = L::TWO ? ci & 1 : 0, buf1 = L::TWO ? buf ^ 1 : 0;   // TWO: the next operand is written beside this one's reads
            __syncthreads();
            const float gn = lin_gate(a, gp, n, time_of(next, l), rev);
            load(next);
            if constexpr (O) {
                f32x4 acc[NVW];
                const int row0 = c * kLinC;
#pragma unroll
                for (int i = 0; i < NVW; ++i) acc[i] = zero4();
                // ---- from earlier chunks
#pragma unroll
                for (int f = 0; f < XF; ++f)
#pragma unroll
                    for (int p = 0; p < NS; ++p)
#pragma unroll
                        for (int i = 0; i < NVW; ++i) {   // consecutive steps: different accumulators
                            const int at = buf * NS * VB * LS + out_col(tile0 + i, m >> 2, m & 3) * LS + 4 * E * f + E * g;
                            acc[i] = X::mma(*reinterpret_cast<const Frag*>(&s.s[p][at]), x[f], acc[i]);
                        }
                // The factors of a step's row: e^{G_16w} and e^{R}; pairs with the 16-step blocks before
                // take theirs in between (the table), so that only the diagonal block forms a factor
                // for each pair.
                const float er = s.eref[w], hi = s.hi[trow], lo = s.lo[trow], es = exp2_hw(hi + lo);
#pragma unroll
                for (int i = 0; i < NVW; ++i) acc[i] = acc[i] * er;
                float dot0 = 0.f, dot1 = 0.f, pd = 0.f;   // r . out from earlier chunks, from all steps before; P's diagonal
                if constexpr (DG) dot0 = rdot(acc, r) * es;
                // ---- pairs of the chunk
                constexpr int NP = JS / 16;
                auto block = [&](int js, auto diagonal) {   // steps JS js .., the last of them w's own
                    constexpr bool D = decltype(diagonal)::value;
                    float p[NP][4];
                    f32x4 pa[NP];
#pragma unroll
                    for (int u = 0; u < NP; ++u) pa[u] = zero4();
#pragma unroll
                    for (int f = 0; f < XF; ++f)
#pragma unroll
                        for (int u = 0; u < NP; ++u)   // a tile past the diagonal is formed too and masked below
                            pa[u] = X::mma(
                                *reinterpret_cast<const Frag*>(&s.y[(16 * (js * NP + u) + m) * LY + 4 * E * f + E * g]),
                                x[f], pa[u]);
#pragma unroll
                    for (int u = 0; u < NP; ++u) {
                        const int jt = js * NP + u;
                        if (!D || jt < w) {
                            const f32x4 f = *reinterpret_cast<const f32x4*>(&s.tab[w - 1][16 * jt + 4 * g]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) p[u][i] = pa[u][i] * (D ? f[i] * es : f[i]);
                        } else {
                            const f32x4 hj = *reinterpret_cast<const f32x4*>(&s.hi[16 * jt + 4 * g]);
                            const f32x4 lj = *reinterpret_cast<const f32x4*>(&s.lo[16 * jt + 4 * g]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int j = 16 * jt + 4 * g + i;
                                const float d = (hi - hj[i]) + (lo - lj[i]);
                                if constexpr (DG) {   // the diagonal apart: it is no part of the gate's gradient
                                    if (j == trow) pd += pa[u][i];
                                    p[u][i] = pa[u][i] * exp2_hw(j < trow ? d : -INFINITY);
                                } else {
                                    p[u][i] = pa[u][i] * exp2_hw(j <= trow ? d : -INFINITY);
                                }
                            }
                        }
                    }
                    constexpr int PP = sizeof(T) == 4 ? 1 : DG ? 3 : 2;   // parts of P
                    Frag pf[PP];
                    if constexpr (PP > 1) {
                        u32x4 part[PP];
#pragma unroll
                        for (int e = 0; e < E; e += 2)
#pragma unroll
                            for (int q = 0; q < PP; ++q) part[q][e / 2] = take_bf16(p[e / 4][e & 3], p[e / 4][(e & 3) + 1]);
#pragma unroll
                        for (int q = 0; q < PP; ++q) pf[q] = __builtin_bit_cast(Frag, part[q]);
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e) pf[0][e] = from_f<T>(p[0][e]);
                    }
                    Frag zf[NVW];
#pragma unroll
                    for (int i = 0; i < NVW; ++i) {
                        const int col0 = sizeof(T) == 2 ? out_col(tile0 + i, m & 3, 0) : out_col(tile0 + i, m >> 2, m & 3);
                        zf[i] = X::load_t(s.z, LZ, js * JS, col0);
                    }
#pragma unroll
                    for (int u = 0; u < PP; ++u)
#pragma unroll
                        for (int i = 0; i < NVW; ++i) acc[i] = X::mma(zf[i], pf[u], acc[i]);
                };
#pragma unroll
                for (int js = 0; js < kLinC / JS; ++js) {   // whole blocks before w's own, then the rest
                    if ((js + 1) * NP <= w) block(js, std::false_type{});
                }
#pragma unroll
                for (int i = 0; i < NVW; ++i) acc[i] = acc[i] * es;
                block(w / NP, std::true_type{});
                if constexpr (DG) {
                    dot1 = rdot(acc, r);
                    pd = sum_lane_groups(pd);
#pragma unroll
                    for (int i = 0; i < NVW; ++i) {
                        const typename Vec4<T>::type z =
                            *reinterpret_cast<const typename Vec4<T>::type*>(&s.z[trow * LZ + out_col(tile0 + i, g, 0)]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][e] += pd * to_f(z[e]);
                    }
                    dot0 = sum_lane_groups(dot0);
                    dot1 = sum_lane_groups(dot1);
                    if constexpr (HV == 1) {
                        const int at = g == 0 ? row_at(trow, 1) / (int)sizeof(T) * 4 : kNowhere;
                        put_dot(0, c, at, dot0);
                        put_dot(1, c, at, dot1);
                    } else if (g == 0) {
                        s.dot[0][half][trow] = dot0;
                        s.dot[1][half][trow] = dot1;
                    }
                }
                // ---- out: 16-byte pieces, 64 consecutive bytes of a step for the four lanes that share it
                const auto ob = lin_range(static_cast<T*>(op.out) + (rows + row0) * a.nd + blk * VB,
                                          (min(n - row0, kLinC) * a.nd - blk * VB) * (int)sizeof(T));
#pragma unroll
                for (int i = 0; i < NVW; i += TP) {
                    const int at = row_at(trow, a.nd) + out_col(tile0 + i, g, 0) * (int)sizeof(T);
                    if constexpr (sizeof(T) == 4) {
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i]), ob, at, 0, 0);
                    } else {
                        u32x2 v[TP];
#pragma unroll
                        for (int u = 0; u < TP; ++u) {
                            typename Vec4<bf16>::type b;
#pragma unroll
                            for (int e = 0; e < 4; ++e) b[e] = (bf16)acc[i + u][e];
                            v[u] = __builtin_bit_cast(u32x2, b);
                        }
                        if constexpr (TP == 2)
                            __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[0][0], v[0][1], v[1][0], v[1][1]}, ob, at, 0, 0);
                        else
                            __builtin_amdgcn_raw_buffer_store_b64(v[0], ob, at, 0, 0);
                    }
                }
            } else if (owns) {
                // ---- state
                if constexpr (DG) {   // the states the gate's gradient is summed from
                    const int e = c / a.snap;
                    if (snap && (rev ? (c + 1) % a.snap == 0 || ci == 0 : c % a.snap == 0) && !(a.nseg > 1 && e == ent0))
                        store_state(snap + e * se, 1.f);
                }
                const float et = s.etot;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[ct] = S[ct] * et;
#pragma unroll
                for (int js = 0; js < kLinC / JS; ++js) {
                    const Frag zf = X::load_t(s.z, LZ, js * JS, 16 * vt + (sizeof(T) == 2 ? 4 * (m & 3) : m));
                    constexpr int ZP = sizeof(T) == 2 ? 3 : 1;   // parts of z e^{..}
                    Frag zw[ZP];
                    if constexpr (ZP == 3) {
                        u32x4 part[ZP];
#pragma unroll
                        for (int e = 0; e < E; e += 2) {
                            const float* ww = &s.ew[js * JS + 16 * (e / 4) + 4 * g + (e & 3)];
                            float u = to_f(zf[e]) * ww[0], v = to_f(zf[e + 1]) * ww[1];
#pragma unroll
                            for (int p = 0; p < ZP; ++p) part[p][e / 2] = take_bf16(u, v);
                        }
#pragma unroll
                        for (int p = 0; p < ZP; ++p) zw[p] = __builtin_bit_cast(Frag, part[p]);
                    } else {
                        const f32x4 ww = *reinterpret_cast<const f32x4*>(&s.ew[js * JS + 4 * g]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) zw[0][i] = zf[i] * ww[i];
                    }
                    Frag yf[CT];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        yf[ct] = X::load_t(s.y, LY, js * JS, 16 * (ct0 + ct) + (sizeof(T) == 2 ? 4 * (m & 3) : m));
#pragma unroll
                    for (int p = 0; p < ZP; ++p)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) S[ct] = X::mma(yf[ct], zw[p], S[ct]);
                }
                if constexpr (OUT && L::TWO) put_state(std::integral_constant<int, NS>{}, buf1);
            }
            if (gates && ci + 1 < count) form_gates(lin_log2(gn, n, time_of(next, l), rev));
            __syncthreads();
            if (gates) put_gates();
            put_tiles();
            if constexpr (OUT && !O && !L::TWO) put_state(std::integral_constant<int, NS>{}, buf1);
            if constexpr (DG && O && HV > 1) {   // the halves of a step's dot
                if (wave < 2) put_dot(wave, c, row_at(l, 1) / (int)sizeof(T) * 4, s.dot[wave][0][l] + s.dot[wave][1][l]);
            }
        };
        // The outputs' waves, which the others wait for, go first (3 % of the time of train steps).
        if constexpr (OUT && O) __builtin_amdgcn_s_setprio(3);
        for (int ci = 0; ci < count; ++ci) chunk(ci);

        // ---- the last state, the segment's own state and factor
        if constexpr (!O) {
            if (!OUT) {
                store_state(snap + ent0 * se, 1.f);
                if (tid == 0 && blk == 0) a.segdec[((long)oi * a.BH + bh) * a.nseg + seg] = exp2_hw((float)dec);
            } else if (rev ? seg == 0 : seg == a.nseg - 1) {
                if (DG && snap) store_state(snap + a.nent * se, 1.f);
                if (op.fin) {   // rev: back through the first step's gate
                    const float g0 = !rev || n == 0 || a.gate == kLinNone ? 0.f : a.gate == kLinHead ? a.g[h] : a.g[rows];
                    store_state(op.fin + bh * se, expf(g0));
                }
            }
        }
    };
    if constexpr (OUT) {
        if (wave < 4 * HV)
            run(std::true_type{});
        else
            run(std::false_type{});
        // steps past the length
        T* o = static_cast<T*>(op.out) + rows * a.nd + blk * VB;
        const int from = max(c0 * kLinC, n), to = min(a.T, c1 * kLinC);
        for (int t = from + tid / PZ; tid < TH / PZ * PZ && t < to; t += TH / PZ)
            *reinterpret_cast<uint4*>(o + (long)t * a.nd + (tid % PZ) * E) = make_uint4(0u, 0u, 0u, 0u);
    } else {
        run(std::false_type{});
    }
}

template <typename T, int KD, int NV> hipError_t lin_launch_nv(const LinArgs& a, int mode, hipStream_t s) {
    const long units = ((long)a.BH * a.nseg + kXcds - 1) / kXcds * kXcds;
    const dim3 grid((unsigned)(units * a.nops * a.nblk)), block(lin_threads(mode, sizeof(T) == 2, NV));
    switch (mode) {
        case kLinState: hipLaunchKernelGGL((lin_kernel<T, KD, NV, kLinState>), grid, block, 0, s, a); break;
        case kLinOut: hipLaunchKernelGGL((lin_kernel<T, KD, NV, kLinOut>), grid, block, 0, s, a); break;
        case kLinDots: hipLaunchKernelGGL((lin_kernel<T, KD, NV, kLinDots>), grid, block, 0, s, a); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <typename T, int KD> hipError_t lin_launch(const LinArgs& a, int nv, int mode, hipStream_t s) {
    switch (nv) {
        case 1: return lin_launch_nv<T, KD, 1>(a, mode, s);
        case 2: return lin_launch_nv<T, KD, 2>(a, mode, s);
        case 4:
            if constexpr (sizeof(T) == 2) return lin_launch_nv<T, KD, 4>(a, mode, s);
            [[fallthrough]];
        default: return hipErrorInvalidValue;
    }
}

}  // namespace dn
