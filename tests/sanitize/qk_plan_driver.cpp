// Exercises the split of the queries' and keys' norms and rotations over workgroups
// (csrc/dn_qk_plan.cpp) over sizes up to the largest integers, without a GPU: the split covers
// every head and token, and what is said to fit does.
#include <climits>
#include <cstdio>
#include <cstring>

#include "dn_qk.h"

static int bad = 0;
#define EXPECT(cond)                                                      \
    do {                                                                  \
        if (!(cond)) {                                                    \
            std::printf("qk plan driver: expectation failed: %s\n", #cond); \
            bad = 1;                                                      \
        }                                                                 \
    } while (0)

int main() {
    const int some[] = {0, 1, 2, 3, 7, 8, 9, 64, 1000, 1 << 20, 1 << 29, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, INT_MAX - 7, INT_MAX};
    const int lens[1] = {0};
    for (int B : some)
        for (int T : some)
            for (int hq : some)
                for (int hk : some)
                    for (int d : {16, 128})
                        for (int kind = 0; kind < 4; ++kind) {
                            if ((long)B * T > 1L << 30) continue;   // refused before the split
                            dn::QkArgs a{};
                            a.B = B, a.T = T, a.d = d, a.norm = 1;
                            a.side[0].heads = hq, a.side[1].heads = hk;
                            const bool fits = dn::qk_fits(a), bwd = kind & 1;
                            const size_t ws = fits ? dn::qk_workspace_bytes(a) : 0;
                            if (kind & 2) a.lens = lens;
                            dn::qk_split(&a, bwd);
                            const long tokens = (long)B * T;
                            EXPECT(a.per >= 1 && a.per <= 8 && a.tiles >= 0 && (a.tiles > 0 || tokens == 0));
                            for (int i = 0; i < 2; ++i) {
                                const long n = a.side[i].heads, g = a.groups[i];
                                EXPECT(g >= 0 && g * a.per >= n && (g - 1) * a.per < (n > 0 ? n : 1));
                            }
                            const long blocks = (long)a.tiles * ((long)a.groups[0] + a.groups[1]);
                            if (fits) EXPECT(blocks < 1L << 24);
                            if (fits && bwd) EXPECT(ws >= (size_t)blocks * d * 4);
                            if (tokens > 0 && (long)hq + hk >= 1L << 30) EXPECT(!fits);
                        }
    if (!bad) std::printf("ok\n");
    return bad;
}
