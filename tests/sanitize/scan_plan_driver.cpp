// Exercises the gated scan's choice of a form and its sizes (csrc/dn_gated_scan_plan.cpp) over shapes up
// to the largest integers, without a GPU: the tiles cover the steps, the strips the channels, and
// every launch, offset and count of what is said to fit is in its kernels' range.
#include <climits>
#include <cstdio>

#include "dn_gated_scan_plan.h"

static int bad = 0;
#define EXPECT(cond)                                                          \
    do {                                                                      \
        if (!(cond)) {                                                        \
            if (!bad) std::printf("scan plan driver: expectation failed: %s (%d %d %d %d)\n", #cond, B, H, T, d); \
            bad = 1;                                                          \
        }                                                                     \
    } while (0)

int main() {
    const int heads[] = {0, 1, 2, 3, 7, 16, 60, 100, 255, 256, 257, 1000, 65537, 1 << 22, 1 << 28, 1 << 30, INT_MAX};
    const int steps[] = {0, 1, 16, 17, 64, 65, 127, 128, 129, 192, 300, 1000, 1024, 1025, 4096, 100000, 1 << 23, 1 << 29, 1 << 30};
    const int widths[] = {1, 2, 3, 5, 16, 31, 48, 63, 64, 65, 67, 100, 128, 1000, 1 << 20, 1 << 21};
    for (int B : heads)
        for (int H : heads)
            for (int T : steps)
                for (int d : widths)
                    for (int bf16 = 0; bf16 < 2; ++bf16) {
                        const dn::GsProblem pr{B, H, T, d, bf16, 0};
                        if (!dn::gs_fits(pr)) {
                            EXPECT((__int128)B * H * ((d + 63) / 64) >= 1 << 22 || (__int128)B * H * d >= 1 << 28);
                            continue;
                        }
                        const size_t states = dn::gs_states_bytes(pr);
                        const size_t sizes[3] = {dn::gs_workspace_bytes(pr, 0), dn::gs_workspace_bytes(pr, 1), dn::gs_workspace_bytes(pr, 2)};
                        EXPECT(sizes[2] >= sizes[0] && sizes[2] >= sizes[1] && sizes[2] >= states);
                        if (B == 0 || H == 0) continue;
                        const long rows = (long)B * H, channels = rows * d;
                        EXPECT(channels < 1L << 28);
                        for (int bwd = 0; bwd < 2; ++bwd) {
                            const dn::GsPlan p = dn::gs_plan(pr, bwd);
                            const long C = 64 / p.groups, wide = p.flat ? (channels + C - 1) / C : rows * ((d + C - 1) / C);
                            EXPECT(p.strips == wide && p.strips > 0);
                            const long run = 16L * p.groups * (p.chain && !bwd ? dn::kGsWavesC : p.waves);
                            EXPECT(p.tiles * run >= T && (T == 0 || (p.tiles - 1) * run < T));
                            EXPECT(T + 16L * 64 < INT_MAX && p.tiles * run < INT_MAX);   // steps of a tile past the end
                            const long blocks = p.chain ? 256 : dn::gs_blocks(p.strips, p.groups);
                            EXPECT(blocks >= (p.chain ? 1 : p.strips) && blocks * 64 * 16 <= 1L << 32);
                            // bytes from a wave's first row to a lane's last: a 31-bit offset
                            const long rowspan = p.flat ? 63 / d + 1 : 0;
                            EXPECT((rowspan * T + 16L * p.groups) * d * 4 < 0x7fffff00L);
                            if (p.chain) {
                                EXPECT(p.groups == 1 && p.strips * p.tiles < 1L << 30 && p.reach >= 1);
                                EXPECT(p.reach <= 8 * (bwd ? dn::kGsWavesB : dn::kGsWavesC));
                                EXPECT(sizes[bwd] >= dn::kGsHead + (size_t)p.strips * p.tiles * dn::kGsMessage);
                                EXPECT(!bwd || 16 * dn::kGsWavesB == dn::kGsSaved);
                            } else if (bwd && p.waves < dn::kGsWavesB) {
                                EXPECT(p.tiles <= 1);
                            }
                        }
                    }
    if (!bad) std::printf("ok\n");
    return bad;
}
