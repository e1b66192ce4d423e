// Exercises the host side of the gated scan's and the queries' and keys' entry points
// (include/dn.h) over sizes up to the largest integers and every kind of refusal, with pointers
// that are never dereferenced; built and run as abi_driver.cpp, without a GPU.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "dn.h"

static int bad = 0;
#define EXPECT(cond)                                                          \
    do {                                                                      \
        if (!(cond)) {                                                        \
            std::printf("scan/qk driver: expectation failed: %s\n", #cond);   \
            bad = 1;                                                          \
        }                                                                     \
    } while (0)

static void* P(uintptr_t i) { return reinterpret_cast<void*>(i << 40); }   // distinct, aligned, never read
static float* F(uintptr_t i) { return reinterpret_cast<float*>(P(i)); }
static int32_t* I(uintptr_t i) { return reinterpret_cast<int32_t*>(P(i)); }

int main() {
    const int some[] = {INT_MIN, -1, 0, 1, 2, 63, 64, 65, 1000, 1 << 20, (1 << 21) + 1, 1 << 30, INT_MAX};
    for (int B : some)
        for (int H : some)
            for (int T : some)
                for (int d : some)
                    for (int dtype = 0; dtype <= 2; ++dtype) {
                        dn_shape s;
                        std::memset(&s, 0, sizeof(s));
                        s.B = B, s.H = H, s.T = T, s.dk = s.dv = d, s.dtype = dtype, s.gate = DN_GATE_VECTOR;
                        const size_t n = dn_gated_scan_states_bytes(&s);
                        const size_t f = dn_gated_scan_workspace_bytes(&s, DN_PASS_FWD);
                        const size_t b = dn_gated_scan_workspace_bytes(&s, DN_PASS_BWD);
                        const size_t r = dn_gated_scan_workspace_bytes(&s, DN_PASS_BWD_RECOMPUTE);
                        EXPECT(r >= n && r >= f && r >= b);
                        EXPECT(dn_gated_scan_workspace_bytes(&s, 3) == 0);
                        // o over x: refused for any size that has elements, or the size itself is
                        const dn_status st = dn_gated_scan_fwd(&s, P(1), F(2), nullptr, nullptr, P(1), nullptr, nullptr, P(9), SIZE_MAX, nullptr);
                        if (B > 0 && H > 0 && T > 0) EXPECT(st != DN_OK && st != DN_ERR_HIP);

                        dn_qk_shape q;
                        std::memset(&q, 0, sizeof(q));
                        q.B = B, q.Hq = q.Hk = H, q.T = T, q.d = 64, q.rot = 32, q.dtype = dtype, q.norm = DN_NORM_L2;
                        q.amplitude = 1.f;
                        for (int64_t* x : {q.q_stride, q.k_stride, q.dq_stride, q.dk_stride}) x[0] = INT64_MAX / 16 * 16, x[1] = d, x[2] = 64;
                        (void)dn_qk_workspace_bytes(&q);
                        const dn_status u = dn_qk_fwd(&q, P(1), P(2), nullptr, nullptr, static_cast<double*>(P(3)), nullptr, nullptr, P(1), P(1), nullptr);
                        if (B > 0 && H > 0 && T > 0) EXPECT(u != DN_OK && u != DN_ERR_HIP);
                    }
    dn_shape s;
    std::memset(&s, 0, sizeof(s));
    s.B = 2, s.H = 3, s.T = 5000, s.dv = 70, s.dtype = DN_BF16, s.gate = DN_GATE_VECTOR, s.flags = DN_FLAG_COUPLED;
    const size_t f = dn_gated_scan_workspace_bytes(&s, DN_PASS_FWD), r = dn_gated_scan_workspace_bytes(&s, DN_PASS_BWD_RECOMPUTE);
    EXPECT(f > 0 && r > f);
    EXPECT(dn_gated_scan_fwd(nullptr, P(1), F(2), nullptr, nullptr, P(3), nullptr, nullptr, P(4), f, nullptr) == DN_ERR_INVALID);
    EXPECT(dn_gated_scan_fwd(&s, P(1), F(2), nullptr, nullptr, P(3), nullptr, nullptr, P(4), f - 1, nullptr) == DN_ERR_WORKSPACE);
    EXPECT(dn_gated_scan_fwd(&s, P(1), F(2), I(3), nullptr, P(3), nullptr, nullptr, P(4), f, nullptr) == DN_ERR_INVALID);
    EXPECT(std::strstr(dn_last_error(), "overlaps") != nullptr);
    EXPECT(dn_gated_scan_bwd(&s, P(1), F(2), nullptr, nullptr, P(3), nullptr, nullptr, P(4), F(5), nullptr, P(6), r - 1, nullptr) == DN_ERR_WORKSPACE);
    EXPECT(dn_gated_scan_bwd(&s, P(1), F(2), nullptr, nullptr, P(3), nullptr, nullptr, P(4), nullptr, nullptr, P(6), r, nullptr) == DN_ERR_INVALID);
    EXPECT(dn_gated_scan_recurrent_fwd(&s, P(1), F(2), nullptr, P(3), nullptr) == DN_ERR_INVALID);
    s.flags = DN_FLAG_NO_SCAN;
    EXPECT(dn_gated_scan_recurrent_fwd(&s, P(1), F(2), F(3), P(4), nullptr) == DN_ERR_INVALID);

    dn_qk_shape q;
    std::memset(&q, 0, sizeof(q));
    q.B = 2, q.Hq = 3, q.Hk = 2, q.T = 5, q.d = 64, q.rot = 64, q.dtype = DN_F32, q.norm = DN_NORM_RMS, q.eps = 1e-6f, q.amplitude = 1.f;
    const int64_t st[3] = {1600, 64, 320};
    for (int64_t* x : {q.q_stride, q.k_stride, q.dq_stride, q.dk_stride}) std::memcpy(x, st, sizeof(st));
    const double* fr = static_cast<double*>(P(5));
    EXPECT(dn_qk_fwd(nullptr, P(1), P(2), F(3), F(4), fr, nullptr, nullptr, P(6), P(7), nullptr) == DN_ERR_INVALID);
    EXPECT(dn_qk_fwd(&q, P(1), P(2), F(3), F(4), nullptr, nullptr, nullptr, P(6), P(7), nullptr) == DN_ERR_INVALID);
    EXPECT(dn_qk_fwd(&q, P(1), P(2), F(3), F(4), fr, I(6), nullptr, P(6), nullptr, nullptr) == DN_ERR_INVALID);
    EXPECT(dn_qk_bwd(&q, P(1), P(2), P(8), P(9), F(3), F(4), fr, nullptr, nullptr, P(10), P(11), F(12), F(13), P(14), 1, nullptr) == DN_ERR_WORKSPACE);
    q.dq_stride[1] = 32;
    EXPECT(dn_qk_bwd(&q, P(1), P(2), P(8), P(9), F(3), F(4), fr, nullptr, nullptr, P(10), P(11), F(12), F(13), P(14), 1 << 20, nullptr) == DN_ERR_INVALID);
    EXPECT(std::strstr(dn_last_error(), "overlap") != nullptr);
    q.eps = NAN;
    EXPECT(dn_qk_workspace_bytes(&q) == 0);
    if (!bad) std::printf("ok\n");
    return bad;
}
