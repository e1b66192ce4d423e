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
// gives a lane 4 NV consecutive channels of one step, S^T four consecutive
// channels of y.  A wave owns 16 steps of the outputs and a share of the state.
//
// Rounding (bf16 I/O): P enters its product with z as two bf16 parts (16 bits: a
// sequence of one step has a single P, whose rounding nothing averages), S is
// rounded once for its product with x, which adds at most as much to an output's
// error as the output's own rounding.  The state itself is held to fp32: its operand
// z e^{..} enters as three bf16 parts (24 bits), since a state (hT, dh0) is an
// fp32 output.  Where the gate's gradient is wanted the state enters the product
// with x in three parts too: that gradient is an fp32 sum of x . S terms.
// fp32 I/O: every product on fp32 matrix-core steps.
#pragma once

#include "dn_device.h"
#include "dn_linear.h"

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

// x as three bf16 parts: x = a + b + c up to 2^-24 of x.
__device__ __forceinline__ void split3(float x, bf16& a, bf16& b, bf16& c) {
    a = (bf16)x;
    const float r = x - (float)a;
    b = (bf16)r;
    c = (bf16)(r - (float)b);
}

template <typename T, int KD, int NV, bool DG> struct LinLds {
    static constexpr int VB = 16 * NV, PAD = 16 / sizeof(T);
    static constexpr int LY = KD + PAD, LZ = VB + PAD;
    static constexpr int NS = DG && sizeof(T) == 2 ? 3 : 1;   // parts of the state operand
    T y[kLinC * LY];
    T z[kLinC * LZ];
    T s[NS][VB * LY];
    // per parity: G (two floats), e^G, e^{G_63 - G}; the chunk's factor
    float hi[2][kLinC], lo[2][kLinC], eg[2][kLinC], ew[2][kLinC], etot[2];
    float rowe[DG ? 4 : 1][DG ? kLinC : 1], colb[DG ? kLinC : 1];
};

// Log-decay (base 2) that the state takes when step t is entered: the step's own
// gate, or with rev that of the step after it; none past the length.  Below -1000 a
// factor is zero in fp32 whatever the rest, so that -inf (a reset) gives no inf - inf.
__device__ __forceinline__ double lin_gate(const LinArgs& a, int bh, int h, int n, int t, int rev) {
    const int at = rev ? t + 1 : t;
    if (a.gate == kLinNone || at >= n || t < 0) return 0.0;
    float g = a.gate == kLinHead ? a.g[h] : a.g[(long)bh * a.T + at];
    g = g < -1000.f ? -1000.f : g;   // NaN stays
    return (double)g * 1.4426950408889634;
}

template <typename T, int KD, int NV, int MODE>
__global__ __launch_bounds__(kLinThreads, 2) void lin_kernel(LinArgs a) {
    constexpr bool OUT = MODE != kLinState, DG = MODE == kLinDots;
    using X = LinT<T>;
    using Frag = typename X::Frag;
    using L = LinLds<T, KD, NV, DG>;
    constexpr int E = X::E, JS = X::JS, VB = 16 * NV, LY = L::LY, LZ = L::LZ, NS = L::NS;
    constexpr int XF = KD / (4 * E);                         // fragments of an x row
    constexpr int WV = 4 / NV;                               // waves that share a state tile column
    constexpr int CT = KD / 16 / WV > 0 ? KD / 16 / WV : 1;  // state tiles of a wave
    constexpr int PY = KD / E, NY = (kLinC * PY + kLinThreads - 1) / kLinThreads;   // 16-byte pieces
    constexpr int PZ = VB / E, NZ = (kLinC * PZ + kLinThreads - 1) / kLinThreads;
    __shared__ __align__(16) L s;

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

    const int tid = threadIdx.x, w = wave_id(), l = lane_id(), g = l >> 4, m = l & 15;
    const int h = bh % a.H, n = lin_len(a.lens, bh / a.H, a.T);
    const int c0 = seg * a.seg_len, c1 = min(a.NT, c0 + a.seg_len);
    const int cv = min(c1, (n + kLinC - 1) / kLinC);   // chunks past it hold no step
    const long rows = (long)bh * a.T;
    const T* xp = static_cast<const T*>(op.x) + rows * a.kd;
    const T* yp = static_cast<const T*>(op.y) + rows * a.kd;
    const T* zp = static_cast<const T*>(op.z) + rows * a.nd + blk * VB;
    const int vt = w % NV, ct0 = (w / NV) * CT;        // this wave's state tiles
    const bool owns = ct0 * 16 < KD;
    const int vrow = blk * VB + 16 * vt + m;           // the state row of this lane

    // ---- state block
    f32x4 S[CT];
    auto each_piece = [&](auto f) {                    // f(tile, offset of its four elements in a state)
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
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) S[ct] = zero4();
    float* snap = op.snap ? op.snap + bh * op.snap_bh : nullptr;
    const long se = (long)a.kd * a.nd;                 // floats of a kept state
    const int ent0 = rev ? (c1 - 1) / a.snap : c0 / a.snap;   // the segment's first entry
    if (OUT && a.nseg > 1) {
        load_state(snap + ent0 * se);
    } else if (OUT && op.init) {
        load_state(op.init + bh * se);
    }
    auto put_state = [&]() {
        if (!OUT || !owns) return;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int at = (16 * vt + m) * LY + 16 * (ct0 + ct) + 4 * g;
            if constexpr (NS == 1) {
                st4<T>(&s.s[0][at], S[ct]);
            } else {
                typename Vec4<bf16>::type p0, p1, p2;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bf16 u0, u1, u2;
                    split3(S[ct][i], u0, u1, u2);
                    p0[i] = u0, p1[i] = u1, p2[i] = u2;
                }
                *reinterpret_cast<typename Vec4<bf16>::type*>(&s.s[0][at]) = p0;
                *reinterpret_cast<typename Vec4<bf16>::type*>(&s.s[1][at]) = p1;
                *reinterpret_cast<typename Vec4<bf16>::type*>(&s.s[2][at]) = p2;
            }
        }
    };

    // ---- loads of a chunk (addresses clamped into the sequence, rows past it zeroed later)
    auto time_of = [&](int c, int row) { return c * kLinC + (rev ? kLinC - 1 - row : row); };
    uint4 yr[NY], zr[NZ];
    Frag xn[XF], x[XF];
    const int trow = 16 * w + m;                       // this lane's step within the chunk
    auto load = [&](int c) {
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int id = tid + kLinThreads * i, t = min(time_of(c, (id / PY) % kLinC), n - 1);
            const int col = (id % PY) * E;
            yr[i] = *reinterpret_cast<const uint4*>(yp + (long)t * a.kd + (col < a.kd ? col : 0));
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
            const int id = tid + kLinThreads * i, t = min(time_of(c, (id / PZ) % kLinC), n - 1);
            zr[i] = *reinterpret_cast<const uint4*>(zp + (long)t * a.nd + (id % PZ) * E);
        }
        if constexpr (OUT) {
            const int t = min(time_of(c, trow), n - 1);
#pragma unroll
            for (int f = 0; f < XF; ++f) {
                const int col = 4 * E * f + E * g;
                xn[f] = *reinterpret_cast<const Frag*>(xp + (long)t * a.kd + (col < a.kd ? col : 0));
            }
        }
    };
    auto put_tiles = [&](int c) {
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int id = tid + kLinThreads * i, row = id / PY, col = (id % PY) * E;
            if (kLinC * PY % kLinThreads == 0 || row < kLinC)
                *reinterpret_cast<uint4*>(&s.y[row * LY + col]) =
                    time_of(c, row) < n && col < a.kd ? yr[i] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
            const int id = tid + kLinThreads * i, row = id / PZ;
            if (kLinC * PZ % kLinThreads == 0 || row < kLinC)
                *reinterpret_cast<uint4*>(&s.z[row * LZ + (id % PZ) * E]) =
                    time_of(c, row) < n ? zr[i] : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (OUT) {
            const bool ok = time_of(c, trow) < n;
#pragma unroll
            for (int f = 0; f < XF; ++f) {
                const uint4 v = __builtin_bit_cast(uint4, xn[f]);
                x[f] = __builtin_bit_cast(Frag, ok && 4 * E * f + E * g < a.kd ? v : make_uint4(0u, 0u, 0u, 0u));
            }
        }
    };
    // running log-decay of a chunk: lane = row, sums in 64 bits (wave 0, which has the
    // fewest pairs under the diagonal)
    double dec = 0.0;                                  // of the run so far
    auto put_gates = [&](double x2, int par) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const double y2 = __shfl_up(x2, d);
            if (l >= d) x2 += y2;
        }
        const double tot = __shfl(x2, 63);
        const float hi = (float)x2, lo = (float)(x2 - (double)hi);
        const float e = exp2_hw(hi);
        s.hi[par][l] = hi;
        s.lo[par][l] = lo;
        s.eg[par][l] = e + e * lo * 0.69314718f;
        s.ew[par][l] = exp2_hw((float)(tot - x2));
        if (l == 63) s.etot[par] = exp2_hw((float)tot);
        dec += tot;
    };

    const int step = rev ? -1 : 1;
    const int first = rev ? cv - 1 : c0, count = cv - c0;
    if (count > 0) {
        load(first);
        if (w == 0) put_gates(lin_gate(a, bh, h, n, time_of(first, l), rev), 0);
        put_tiles(first);
        put_state();
    }
    int par = 0;
    for (int ci = 0; ci < count; ++ci, par ^= 1) {
        const int c = first + step * ci;
        const bool more = ci + 1 < count;
        __syncthreads();
        double gn = 0.0;
        if (more) {
            load(c + step);
            if (w == 0) gn = lin_gate(a, bh, h, n, time_of(c + step, l), rev);
        }
        if constexpr (DG) {   // the states the gate's gradient is summed from
            const int e = c / a.snap;
            if (snap && (rev ? (c + 1) % a.snap == 0 || ci == 0 : c % a.snap == 0) && !(a.nseg > 1 && e == ent0))
                store_state(snap + e * se, 1.f);
        }
        f32x4 acc[NV];
        if constexpr (OUT) {
            const int tt = time_of(c, trow);
            // rows of the other factor of the gate's gradient, 4 NV channels of this lane's step
            T r[DG ? 4 * NV : 1];
            float dot = 0.f, col = 0.f;
            if constexpr (DG) {
                const T* rp = static_cast<const T*>(op.r) + (rows + min(tt, n - 1)) * a.nd + blk * VB + 4 * NV * g;
                typedef typename Vec4<T>::type V4;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const V4 v = *reinterpret_cast<const V4*>(rp + 4 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[4 * i + e] = tt < n ? (T)v[e] : (T)0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) acc[i] = zero4();
            // ---- from earlier chunks
#pragma unroll
            for (int f = 0; f < XF; ++f)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int at = (4 * NV * (m >> 2) + 4 * i + (m & 3)) * LY + 4 * E * f + E * g;
#pragma unroll
                    for (int p = 0; p < NS; ++p)
                        acc[i] = X::mma(*reinterpret_cast<const Frag*>(&s.s[p][at]), x[f], acc[i]);
                }
            const float eg = s.eg[par][trow];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                acc[i] = acc[i] * eg;
                if constexpr (DG) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) dot += acc[i][e] * to_f(r[4 * i + e]);
                }
            }
            // ---- pairs of the chunk
            const float hi = s.hi[par][trow], lo = s.lo[par][trow];
            constexpr int NP = JS / 16;
#pragma unroll
            for (int js = 0; js < kLinC / JS; ++js) {
                if (js * NP > w) continue;
                float p[NP][4];
#pragma unroll
                for (int u = 0; u < NP; ++u) {
                    const int jt = js * NP + u;
                    if (jt > w) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[u][i] = 0.f;
                        continue;
                    }
                    f32x4 pa = zero4();
#pragma unroll
                    for (int f = 0; f < XF; ++f)
                        pa = X::mma(*reinterpret_cast<const Frag*>(&s.y[(16 * jt + m) * LY + 4 * E * f + E * g]), x[f], pa);
                    const f32x4 hj = *reinterpret_cast<const f32x4*>(&s.hi[par][16 * jt + 4 * g]);
                    const f32x4 lj = *reinterpret_cast<const f32x4*>(&s.lo[par][16 * jt + 4 * g]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = 16 * jt + 4 * g + i;
                        const float d = (hi - hj[i]) + (lo - lj[i]);
                        p[u][i] = pa[i] * exp2_hw(j <= trow ? d : -INFINITY);
                    }
                    if constexpr (DG) {
                        if (op.role == 2) {   // E = P o (r z^T), summed along both axes
                            f32x4 q = zero4();
                            const T* zr_ = &s.z[(16 * jt + m) * LZ + 4 * NV * g];
                            if constexpr (4 * NV >= E) {
#pragma unroll
                                for (int f = 0; f < 4 * NV / E; ++f) {
                                    Frag rb;
#pragma unroll
                                    for (int e = 0; e < E; ++e) rb[e] = r[E * f + e];
                                    q = X::mma(*reinterpret_cast<const Frag*>(zr_ + E * f), rb, q);
                                }
                            } else {   // 16 channels of bf16: half of the K slots are zero
                                Frag za, rb;
                                const typename Vec4<T>::type v = *reinterpret_cast<const typename Vec4<T>::type*>(zr_);
#pragma unroll
                                for (int e = 0; e < E; ++e) {
                                    za[e] = e < 4 ? (T)v[e & 3] : (T)0.f;
                                    rb[e] = e < 4 ? r[e & 3] : (T)0.f;
                                }
                                q = X::mma(za, rb, q);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int j = 16 * jt + 4 * g + i;
                                const float e = j == trow ? 0.f : p[u][i] * q[i];   // the diagonal cancels
                                col += e;
                                const float rs = row16_sum(e);
                                if (m == 0) s.rowe[w][j] = rs;
                            }
                        }
                    }
                }
                constexpr int PP = sizeof(T) == 2 ? 2 : 1;   // parts of P
                Frag pf[PP];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float v = p[e / 4][e & 3];
                    pf[0][e] = from_f<T>(v);
                    if constexpr (PP == 2) pf[1][e] = from_f<T>(v - to_f(pf[0][e]));
                }
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int col0 = sizeof(T) == 2 ? 4 * NV * (m & 3) + 4 * i : 4 * NV * (m >> 2) + 4 * i + (m & 3);
                    const Frag zf = X::load_t(s.z, LZ, js * JS, col0);
#pragma unroll
                    for (int u = 0; u < PP; ++u) acc[i] = X::mma(zf, pf[u], acc[i]);
                }
            }
            // ---- out: 4 NV consecutive channels of one step
            if (tt < a.T) {
                T* o = static_cast<T*>(op.out) + (rows + tt) * a.nd + blk * VB + 4 * NV * g;
                const bool ok = tt < n;
#pragma unroll
                for (int i = 0; i < NV; ++i) st4<T>(o + 4 * i, ok ? acc[i] : zero4());
            }
            if constexpr (DG) {
                if (op.role == 1) {
                    dot = sum_lane_groups(dot);
                    if (g == 0 && tt < n) op.dots[((long)blk * a.BH + bh) * a.T + tt] = dot;
                } else {
                    dot = sum_lane_groups(dot + col);
                    if (g == 0) s.colb[trow] = dot;
                }
            }
        }
        // ---- state
        if (owns) {
            const float et = s.etot[par];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[ct] = S[ct] * et;
#pragma unroll
            for (int js = 0; js < kLinC / JS; ++js) {
                const Frag zf = X::load_t(s.z, LZ, js * JS, 16 * vt + (sizeof(T) == 2 ? 4 * (m & 3) : m));
                Frag zw[sizeof(T) == 2 ? 3 : 1];
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const f32x4 ww = *reinterpret_cast<const f32x4*>(&s.ew[par][js * JS + 16 * q + 4 * g]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = to_f(zf[4 * q + i]) * ww[i];
                        if constexpr (sizeof(T) == 2) {
                            bf16 u0, u1, u2;
                            split3(v, u0, u1, u2);
                            zw[0][4 * q + i] = u0, zw[1][4 * q + i] = u1, zw[2][4 * q + i] = u2;
                        } else {
                            zw[0][i] = v;
                        }
                    }
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const Frag yf = X::load_t(s.y, LY, js * JS, 16 * (ct0 + ct) + (sizeof(T) == 2 ? 4 * (m & 3) : m));
                    S[ct] = X::mma(yf, zw[0], S[ct]);
                    if constexpr (sizeof(T) == 2) {
                        if (a.gate != kLinNone) {   // without a gate the first part is all of z
                            S[ct] = X::mma(yf, zw[1], S[ct]);
                            S[ct] = X::mma(yf, zw[2], S[ct]);
                        }
                    }
                }
            }
        }
        if (w == 0 && more) put_gates(gn, par ^ 1);
        __syncthreads();
        if constexpr (DG) {
            const int row = tid, tt = time_of(c, row & (kLinC - 1));
            if (op.role == 2 && row < kLinC && tt < n) {
                float d = -s.colb[row];
                for (int u = row / 16; u < 4; ++u) d += s.rowe[u][row];
                op.dots[((long)blk * a.BH + bh) * a.T + tt] = d;
            }
        }
        if (more) {
            put_tiles(c + step);
            put_state();
        }
    }

    // ---- what is left: steps past the length, the last state, the segment's factor
    if constexpr (OUT) {
        T* o = static_cast<T*>(op.out) + rows * a.nd + blk * VB;
        const int from = max(c0, cv) * kLinC, to = min(a.T, c1 * kLinC);
        for (int t = from + tid / PZ; t < to; t += kLinThreads / PZ)
            *reinterpret_cast<uint4*>(o + (long)t * a.nd + (tid % PZ) * E) = make_uint4(0u, 0u, 0u, 0u);
        if (rev ? seg == 0 : seg == a.nseg - 1) {
            if (DG && !rev && snap) store_state(snap + a.nent * se, 1.f);
            if (op.fin) {   // rev: back through the first step's gate
                const float g0 = !rev || n == 0 || a.gate == kLinNone ? 0.f : a.gate == kLinHead ? a.g[h] : a.g[rows];
                store_state(op.fin + bh * se, expf(g0));
            }
        }
    } else {
        store_state(snap + ent0 * se, 1.f);
        if (tid == 0 && blk == 0) a.segdec[((long)oi * a.BH + bh) * a.nseg + seg] = exp2_hw((float)dec);
    }
}

template <typename T, int KD, int NV> hipError_t lin_launch_nv(const LinArgs& a, int mode, hipStream_t s) {
    const long units = ((long)a.BH * a.nseg + kXcds - 1) / kXcds * kXcds;
    const dim3 grid((unsigned)(units * a.nops * a.nblk)), block(kLinThreads);
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
