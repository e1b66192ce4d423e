// dn_tree_kernels.h -- the nodes of a tree of drafted tokens read from one state.
//
// Node n hangs on parent p(n) < n or on the root, whose state S is the sequence's.
// With Gam_n the log-decays summed along the path to n and "anc" the nodes on that path
// before n, the states of all nodes unroll to
//     u_n = beta_n (v_n - S e^{Gam_n} k_n - sum_{m anc n} u_m (k_m . e^{Gam_n - Gam_m} k_n))
//     o_n = S e^{Gam_n} q_n + sum_{m anc n or m = n} u_m (k_m . e^{Gam_n - Gam_m} q_n)
// (linear attention: u_n = v_n): one triangular system whose mask is the tree's, so the
// state is read once whatever the number of branches, and never copied.
//
// A workgroup takes one (b, h) and a block of state rows (16 a wave).  Everything is held
// to fp32, since u is an fp32 output from which states are continued: fp32 matrix-core
// steps for fp32 keys and queries; for bf16 ones bf16 steps that are as exact, on three
// bf16 parts (24 bits) of the state and of keys and queries scaled by channel gates: a
// fifth of the fp32 steps' time, 0.4 of it with channel gates.
// The state's operands come straight from its rows.  A wave keeps its
// columns of u in accumulators from the first product to the last: accumulator row
// 4 g + i is K slot g of step i of the next product, so the chain X -> R -> u -> o needs
// no LDS besides the node-by-node matrices.  The system is solved by 16-node blocks, the
// diagonal ones inverted by substitution, one lane a column.
//
// Measured (bf16, d = 128, whole calls): 64 x 16 heads, 16 nodes 23 us for 92 MB (the kernel
// 20: 4.6 TB/s where a copy reaches 5.2, bound by the state's bytes; fp32 29); 16 x 16 heads, 61
// nodes with channel gates 31.5 us for 49 MB (fp32 35): one workgroup on a compute unit, bound
// by its chain of phases (loads, path sums, scaling, products, solution), the products a third
// of it.  With a path's |Gam| beyond 60, where each node's path is walked by a wave: the same trees
// 50 us, chains of 61 nodes 142.
#pragma once

#include <type_traits>

#include "dn.h"
#include "dn_device.h"
#include "dn_split.h"
#include "dn_tree.h"

namespace dn {

__device__ __forceinline__ f32x4 tree_mma(f32x4 a, f32x4 b, f32x4 c) {   // K over 4 g + i
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// Eight floats as three bf16 parts (24 bits).
__device__ __forceinline__ void tree_parts(f32x4 a, f32x4 b, bf16x8 (&p)[3]) {
    float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    unsigned u[3][4];
#pragma unroll
    for (int e = 0; e < 8; e += 2)
#pragma unroll
        for (int r = 0; r < 3; ++r) u[r][e / 2] = take_bf16(x[e], x[e + 1]);
#pragma unroll
    for (int r = 0; r < 3; ++r) p[r] = *reinterpret_cast<const bf16x8*>(u[r]);
}

// Gates below -1000 are a factor of zero whatever follows, and their sums stay finite.
__device__ __forceinline__ float tree_clamp(float g) { return g < -1000.f ? -1000.f : g; }

// Lane n: the node's parent (-1: the root; an index that is no earlier node counts as the
// root), by the first n nodes of the tree.
__device__ __forceinline__ int tree_parent(const int* parent, int count, int n) {
    const int p = n < count ? parent[n] : -1;
    return p >= 0 && p < n ? p : -1;
}
// Lane n of a whole wave: the nodes on its path (itself included) as bits, and x summed
// along it, by pointer doubling.
template <int NP> __device__ __forceinline__ unsigned long long tree_path(int p, int n, double& x) {
    unsigned long long on = 1ull << n;
#pragma unroll
    for (int r = 1; r < NP; r *= 2) {   // NP nodes: a path of at most NP
        const int from = p < 0 ? n : p;
        const unsigned long long o = __shfl(on, from);
        const double y = __shfl(x, from);
        const int pp = __shfl(p, from);
        if (p >= 0) {
            on |= o;
            x += y;
            p = pp;
        }
    }
    return on;
}

template <typename T, int DK, int NP, bool VEC> struct TreeLds {
    static constexpr bool BF = sizeof(T) == 2, PARTS = BF && VEC;
    static constexpr int DP = BF && DK < 32 ? 32 : DK;     // one bf16 step at least, zeros behind DK
    static constexpr int LD = DK + 4, LN = NP + 4;
    static constexpr int KP = PARTS ? 3 : 1;               // of k and q; per channel gate: times e^{Gam}.  bf16 parts or fp32
    static constexpr int LX = BF ? DP + (VEC ? 8 : 16) : LD;
    typedef typename std::conditional<BF, bf16, float>::type X;
    __align__(16) X kx[KP][NP][LX];
    static constexpr int ROOM = (int)(2 * sizeof(float) * LN - sizeof(X) * KP * LX) * NP;
    char room[PARTS && ROOM > 0 ? ROOM : 16];   // of A and P behind kx (see sys)
    X qx[KP][NP][LX];
    float km[VEC ? NP : 1][VEC ? LD : 1];   // k e^{-Gam}, or the gates where that would overflow
    // The system's matrix A (its diagonal blocks inverted in place) and the outputs' P.  PARTS: where kx
    // lies, which is read no more when they are written (the third part of q has its room from that).
    float sys[PARTS ? 1 : 2][PARTS ? 1 : NP][PARTS ? 1 : LN];
    unsigned long long on[NP];
    double gam[NP];                      // Gam of a gate per step or head
    float beta[NP];
    int parent[NP];
    float low[8];                        // less the largest |Gam| of any channel, by wave
};

template <typename T, int DK, int NP, int NW, bool VEC>
__global__ __launch_bounds__(64 * NW, NP == 16 && !VEC ? 8 : 2) void tree_kernel(TreeArgs a) {
    using L = TreeLds<T, DK, NP, VEC>;
    constexpr bool BF = L::BF, PARTS = L::PARTS;
    constexpr int KP = L::KP;
    constexpr int TH = 64 * NW, NT = NP / 16, F = DK / 16, Q = DK / 4;
    __shared__ __align__(16) L s;
    typedef float Sys[NP][L::LN];
    Sys* sys = reinterpret_cast<Sys*>(PARTS ? static_cast<void*>(s.kx) : static_cast<void*>(s.sys));
    Sys &A = sys[0], &P = sys[1];
    const int nblk = (a.dv / 16 + NW - 1) / NW;
    const int BH = a.B * a.H;
    int bh, blk;   // blocks of a head: ids equal mod 8 (one XCD, whose L2 holds its rows)
    head_and_block(nblk, BH, bh, blk);
    const int b = bh / a.H, h = bh % a.H, N = a.N;
    const int tid = threadIdx.x, l = lane_id(), g = l >> 4, m = l & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int cnt = a.counts ? a.counts[b] : N;
    cnt = __builtin_amdgcn_readfirstlane(cnt < 0 ? 0 : cnt > N ? N : cnt);
    const bool delta = a.beta != nullptr;
    const int tile = blk * NW + wave;
    const bool active = 16 * tile < a.dv;
    const long rows = (long)bh * N;

    // ---- loads, first needed first: the tree, keys and queries, then the state's rows in the
    // order their products take them
    int p = -1;
    double gate = 0.0;
    if (wave == 0) {
        p = l < NP ? tree_parent(a.parent + (long)b * N, cnt, l) : -1;
        if (l < cnt && a.gate == DN_GATE_SCALAR) gate = tree_clamp(a.g[rows + l]);
        if (l < cnt && a.gate == DN_GATE_HEAD) gate = tree_clamp(a.g[h]);
    }
    constexpr int PC = (NP * Q + TH - 1) / TH;   // pieces of four channels a thread
    f32x4 kr[PC], qr[PC], gr[VEC ? PC : 1];
    float br[PC];
#pragma unroll
    for (int i = 0; i < PC; ++i) {
        const int id = tid + TH * i, n = id / Q, c = 4 * (id % Q);
        kr[i] = qr[i] = zero4();
        br[i] = 0.f;
        if constexpr (VEC) gr[i] = zero4();
        if (n < cnt) {
            const long at = (rows + n) * DK + c;
            if constexpr (VEC) gr[i] = *reinterpret_cast<const f32x4*>(a.g + at);
            kr[i] = ld4<T>(static_cast<const T*>(a.k) + at);
            qr[i] = ld4<T>(static_cast<const T*>(a.q) + at);
            if (delta && c == 0) br[i] = a.beta[rows + n];
        }
    }
    constexpr int SF = L::DP / 16;
    f32x4 S[SF];   // pieces of four channels: of step f, 16 f + 4 g; BF: of step f / 2, 32 (f / 2) + 8 g + 4 (f % 2)
    const int vrow = 16 * tile + m;
#pragma unroll
    for (int f = 0; f < SF; ++f) {
        const int c = BF ? 32 * (f / 2) + 8 * g + 4 * (f % 2) : 16 * f + 4 * g;
        S[f] = active && c < DK ? *reinterpret_cast<const f32x4*>(a.state + ((long)bh * a.dv + vrow) * DK + c) : zero4();
    }

    // ---- the tree: paths and their decays
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            const int id = tid + TH * i;
            if (id < NP * Q)
                *reinterpret_cast<f32x4*>(&s.km[id / Q][4 * (id % Q)]) =
                    f32x4{tree_clamp(gr[i][0]), tree_clamp(gr[i][1]), tree_clamp(gr[i][2]), tree_clamp(gr[i][3])};
        }
    }
    if (wave == 0) {
        const unsigned long long on = tree_path<NP>(p, l, gate);
        if (l < NP) {
            s.on[l] = on;
            s.gam[l] = gate;
            s.parent[l] = p;
        }
    }
    bool deep = false;
    float* G0 = reinterpret_cast<float*>(PARTS ? static_cast<void*>(s.kx) : static_cast<void*>(s.qx));   // Gam of every channel
    constexpr int LD = L::LD;
    if constexpr (VEC) {
        __syncthreads();
        // path sums of every channel: the paths' 0/1 matrix times the gates
        float low = 0.f;
        for (int ct = wave; ct < F; ct += NW) {
            f32x4 G[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) G[t] = zero4();
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                f32x4 gv;
#pragma unroll
                for (int i = 0; i < 4; ++i) gv[i] = s.km[16 * q + 4 * g + i][16 * ct + m];
#pragma unroll
                for (int t = q; t < NT; ++t) {   // paths hold earlier nodes only
                    const unsigned bits = (unsigned)(s.on[16 * t + m] >> (16 * q + 4 * g));
                    const f32x4 on = {(float)(bits & 1), (float)(bits >> 1 & 1), (float)(bits >> 2 & 1), (float)(bits >> 3 & 1)};
                    G[t] = tree_mma(on, gv, G[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    G0[(16 * t + 4 * g + i) * LD + 16 * ct + m] = G[t][i];
                    low = fminf(low, -fabsf(G[t][i]));
                }
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) low = fminf(low, __shfl_xor(low, d));
        if (l == 0) s.low[wave] = low;
        __syncthreads();
        // Up to |Gam| = 60 e^{Gam}, e^{-Gam} and their parts keep clear of the ends of the
        // exponents' range; beyond, the pairs' decays are formed one by one.
#pragma unroll
        for (int u = 0; u < NW; ++u) deep |= s.low[u] < -60.f;
    }

    // ---- keys and queries to LDS; the keys' square norms for Kaczmarz steps
#pragma unroll
    for (int j = 0; j < PC; ++j) {
        const int id = tid + TH * j, n = id / Q, c = 4 * (id % Q);
        if (NP * Q % TH != 0 && id >= NP * Q) continue;   // whole waves
        const f32x4 kk = kr[j];
        const float norm = group_sum<Q>(kk[0] * kk[0] + kk[1] * kk[1] + kk[2] * kk[2] + kk[3] * kk[3]);
        if (c == 0) s.beta[n] = a.kz && n < cnt ? br[j] / (norm + a.eps) : br[j];
        if constexpr (VEC) {
            f32x4 e = zero4(), r = zero4();
            if (n < cnt) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(&G0[n * LD + c]);
                r = *reinterpret_cast<const f32x4*>(&s.km[n][c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e[i] = expf(x[i]);
                    if (!deep) r[i] = kk[i] * expf(-x[i]);
                }
            }
            *reinterpret_cast<f32x4*>(&s.km[n][c]) = r;
            kr[j] = kk * e;
            qr[j] = qr[j] * e;
        }
    }
    if constexpr (PARTS) __syncthreads();   // the path sums lie where the parts go
#pragma unroll
    for (int j = 0; j < PC; ++j) {
        const int id = tid + TH * j, n = id / Q, c = 4 * (id % Q);
        if (NP * Q % TH != 0 && id >= NP * Q) continue;
        f32x4 kk = kr[j], qq = qr[j];
        auto put = [&](typename L::X (&to)[NP][L::LX], f32x4 (&v)) {   // the first part; what it leaves stays in v
            if constexpr (BF) {
                float v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
                const unsigned u0 = take_bf16(v0, v1), u1 = take_bf16(v2, v3);
                *reinterpret_cast<uint2*>(&to[n][c]) = make_uint2(u0, u1);
                v = f32x4{v0, v1, v2, v3};
                if constexpr (L::DP > DK) *reinterpret_cast<uint2*>(&to[n][DK + c]) = make_uint2(0u, 0u);
            } else {
                *reinterpret_cast<f32x4*>(&to[n][c]) = v;
            }
        };
#pragma unroll
        for (int r = 0; r < KP; ++r) put(s.kx[r], kk);
#pragma unroll
        for (int r = 0; r < KP; ++r) put(s.qx[r], qq);
    }
    __syncthreads();

    // ---- S k_n and S q_n of every node, rows n, columns the wave's state rows
    f32x4 X[NT], o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) X[t] = zero4(), o[t] = zero4();
    // Parts r of one factor and q of the other are multiplied for r + q < 3.
    if (active) {
        if constexpr (BF) {
#pragma unroll
            for (int f = 0; f < L::DP / 32; ++f) {
                bf16x8 sp[3];
                tree_parts(S[2 * f], S[2 * f + 1], sp);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int r = 0; r < KP; ++r) {
                        const bf16x8 qf = *reinterpret_cast<const bf16x8*>(&s.qx[r][16 * t + m][32 * f + 8 * g]);
#pragma unroll
                        for (int q = 0; q < 3 - r; ++q)
                            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf, sp[q], o[t], 0, 0, 0);
                    }
                    if (!delta) continue;
#pragma unroll
                    for (int r = 0; r < KP; ++r) {
                        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(&s.kx[r][16 * t + m][32 * f + 8 * g]);
#pragma unroll
                        for (int q = 0; q < 3 - r; ++q)
                            X[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, sp[q], X[t], 0, 0, 0);
                    }
                }
            }
        } else {
#pragma unroll
            for (int f = 0; f < F; ++f) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    o[t] = tree_mma(*reinterpret_cast<const f32x4*>(&s.qx[0][16 * t + m][16 * f + 4 * g]), S[f], o[t]);
                    if (delta)
                        X[t] = tree_mma(*reinterpret_cast<const f32x4*>(&s.kx[0][16 * t + m][16 * f + 4 * g]), S[f], X[t]);
                }
            }
        }
    }
    float vin[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 16 * t + 4 * g + i;
            vin[t][i] = active && n < cnt ? to_f(static_cast<const T*>(a.v)[(rows + n) * a.dv + vrow]) : 0.f;
        }

    // ---- node by node: A = beta (k_n . e^{..} k_m) for m before n on its path, P with q_n, m = n too
    constexpr int TRI = NT * (NT + 1) / 2, TILES = (2 * TRI + NW - 1) / NW;   // of both; of a wave
    if (!deep) {
        f32x4 pair[TILES];
        int row[TILES], col[TILES];   // tiles of nodes
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
            const int id = wave + NW * j;
            const bool isP = id < TRI;
            int tn = 0, tm = isP ? id : id - TRI;
            while (tm > tn) tm -= ++tn;
            row[j] = tn, col[j] = tm;
            pair[j] = zero4();
            if (id >= (delta ? 2 : 1) * TRI) continue;
            f32x4 acc = zero4();
            if constexpr (BF) {
#pragma unroll
                for (int f = 0; f < L::DP / 32; ++f) {
                    bf16x8 mp[3];
                    if constexpr (VEC) {   // k e^{-Gam} of 8 channels in parts (zero behind DK)
                        const int c = 32 * f + 8 * g;
                        const float* mr = &s.km[16 * tm + m][c < DK ? c : 0];
                        const f32x4 z = zero4();
                        tree_parts(c < DK ? *reinterpret_cast<const f32x4*>(mr) : z,
                                   c < DK ? *reinterpret_cast<const f32x4*>(mr + 4) : z, mp);
                    } else {
                        mp[0] = *reinterpret_cast<const bf16x8*>(&s.kx[0][16 * tm + m][32 * f + 8 * g]);
                    }
#pragma unroll
                    for (int r = 0; r < KP; ++r) {
                        const bf16x8 nf = *reinterpret_cast<const bf16x8*>(
                            isP ? &s.qx[r][16 * tn + m][32 * f + 8 * g] : &s.kx[r][16 * tn + m][32 * f + 8 * g]);
#pragma unroll
                        for (int q = 0; q < KP - r; ++q)
                            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(nf, mp[q], acc, 0, 0, 0);
                    }
                }
            } else {
                const float* nr = isP ? &s.qx[0][16 * tn + m][0] : &s.kx[0][16 * tn + m][0];
                const float* mr = VEC ? &s.km[16 * tm + m][0] : &s.kx[0][16 * tm + m][0];
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc = tree_mma(*reinterpret_cast<const f32x4*>(nr + 16 * f + 4 * g),
                                   *reinterpret_cast<const f32x4*>(mr + 16 * f + 4 * g), acc);
            }
            pair[j] = acc;
        }
        if constexpr (PARTS) __syncthreads();   // kx is read no more
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
            const int id = wave + NW * j;
            const bool isP = id < TRI;
            if (id >= (delta ? 2 : 1) * TRI) continue;
            const int mm = 16 * col[j] + m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = 16 * row[j] + 4 * g + i;
                const bool on = (s.on[n] >> mm & 1) && (isP || mm != n);
                float w = 1.f;
                if (!VEC) w = __builtin_amdgcn_exp2f((float)((s.gam[n] - s.gam[mm]) * 1.4426950408889634));
                const float x = on ? pair[j][i] * w : 0.f;
                if (isP) P[n][mm] = x;
                else A[n][mm] = x * s.beta[n];
            }
        }
    } else if constexpr (VEC) {
        // Up each node's path with the decay of the nodes passed, a wave a node.
        if constexpr (PARTS) __syncthreads();   // kx is read no more
        for (int id = tid; id < NP * NP; id += TH) A[id / NP][id % NP] = 0.f, P[id / NP][id % NP] = 0.f;
        __syncthreads();
        constexpr int C = (DK + 63) / 64;
        for (int n = wave; n < cnt; n += NW) {
            float kn[C], qn[C], w[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const bool in = l + 64 * c < DK;
                const long at = (rows + n) * DK + (in ? l + 64 * c : 0);
                kn[c] = in ? to_f(static_cast<const T*>(a.k)[at]) : 0.f;
                qn[c] = in ? to_f(static_cast<const T*>(a.q)[at]) : 0.f;
                w[c] = 0.f;
            }
            const float bn = s.beta[n];
            for (int mm = n; mm >= 0; mm = s.parent[mm]) {
                float pk = 0.f, pq = 0.f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int ch = l + 64 * c < DK ? l + 64 * c : 0;
                    const float x = to_f(static_cast<const T*>(a.k)[(rows + mm) * DK + ch]) * expf(w[c]);
                    pk += x * kn[c];
                    pq += x * qn[c];
                    w[c] += s.km[mm][ch];
                }
#pragma unroll
                for (int d = 1; d < 64; d *= 2) pk += __shfl_xor(pk, d), pq += __shfl_xor(pq, d);
                if (l == 0) {
                    P[n][mm] = pq;
                    if (mm != n && delta) A[n][mm] = bn * pk;
                }
            }
        }
    }
    __syncthreads();

    // ---- diagonal blocks of I + A inverted in place: lane j a column, by substitution
    if (delta) {
        if (tid < NP) {
            const int r0 = tid & ~15, j = tid & 15;
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x = i == j ? 1.f : 0.f;
#pragma unroll
                for (int q = 0; q < i; ++q) x -= A[r0 + i][r0 + q] * t[q];
                t[i] = x;
            }
            __builtin_amdgcn_wave_barrier();   // every lane of the block has read it
#pragma unroll
            for (int i = 0; i < 16; ++i) A[r0 + i][r0 + j] = t[i];
        }
        __syncthreads();
    }
    if (!active) return;

    // ---- R = beta (v - S e^{Gam} k), u block by block, then the outputs
    f32x4 u[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        f32x4 eg, r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 16 * t + 4 * g + i;
            eg[i] = VEC ? 1.f : __builtin_amdgcn_exp2f((float)(s.gam[n] * 1.4426950408889634));
            r[i] = delta ? s.beta[n] * (vin[t][i] - eg[i] * X[t][i]) : vin[t][i];
        }
        o[t] = o[t] * eg;
        if (delta) {
            f32x4 sub = zero4();
#pragma unroll
            for (int q = 0; q < t; ++q) sub = tree_mma(*reinterpret_cast<const f32x4*>(&A[16 * t + m][16 * q + 4 * g]), u[q], sub);
            r = r - sub;
            u[t] = tree_mma(*reinterpret_cast<const f32x4*>(&A[16 * t + m][16 * t + 4 * g]), r, zero4());
        } else {
            u[t] = r;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q <= t; ++q) o[t] = tree_mma(*reinterpret_cast<const f32x4*>(&P[16 * t + m][16 * q + 4 * g]), u[q], o[t]);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 16 * t + 4 * g + i;
            if (n >= N) continue;
            const long at = (rows + n) * a.dv + vrow;
            static_cast<T*>(a.o)[at] = from_f<T>(n < cnt ? o[t][i] : 0.f);
            if (a.u) a.u[at] = n < cnt ? u[t][i] : 0.f;
        }
}

template <typename T, int DK, int NP, int NW> hipError_t tree_launch_np(const TreeArgs& a, hipStream_t s) {
    const int nblk = (a.dv / 16 + NW - 1) / NW;
    const dim3 grid((unsigned)((long)a.B * a.H * nblk)), block(64 * NW);
    if (a.gate == DN_GATE_VECTOR)
        hipLaunchKernelGGL((tree_kernel<T, DK, NP, NW, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((tree_kernel<T, DK, NP, NW, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

// Eight waves, 128 state rows, share the node-by-node products and the staged rows (64
// rows a workgroup: 35.8 us against 34.1 at 64 x 16 heads, 16 nodes); at 16 nodes 64
// registers then let all of a compute unit's workgroups of such a batch run at once
// (34.1 -> 24.7 us; with the bf16 steps 20).
template <typename T, int DK> hipError_t tree_launch_dk(const TreeArgs& a, hipStream_t s) {
    if (a.N <= 16) return tree_launch_np<T, DK, 16, 8>(a, s);
    if (a.N <= 32) return tree_launch_np<T, DK, 32, 8>(a, s);
    return tree_launch_np<T, DK, 64, 8>(a, s);
}

template <typename T> hipError_t tree_launch(const TreeArgs& a, hipStream_t s) {
    switch (a.dk) {
        case 16: return tree_launch_dk<T, 16>(a, s);
        case 32: return tree_launch_dk<T, 32>(a, s);
        case 64: return tree_launch_dk<T, 64>(a, s);
        case 128: return tree_launch_dk<T, 128>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace dn
