// The wait of csrc/dn_wait.h on the host: for what is there, what comes, and what never does.
#include <cstdio>

#include "dn_wait.h"

static int bad = 0;
#define EXPECT(cond)                                                    \
    do {                                                                \
        if (!(cond)) {                                                  \
            std::printf("wait driver: expectation failed: %s\n", #cond); \
            bad = 1;                                                    \
        }                                                               \
    } while (0)

// Looks, `limit` at most, until a message that comes with look number `comes` (-1: never); how many it took,
// and whether it was given up.
static long looks(long comes, int limit, bool* lost) {
    long n = 0;
    *lost = false;
    dn::wait_until([&] { return *lost || (comes >= 0 && n >= comes); }, [&] { ++n; }, [&] { *lost = true; }, limit);
    return n;
}

int main() {
    bool lost;
    for (int limit : {1, 2, 1000, 1 << 20}) {
        EXPECT(looks(0, limit, &lost) == 0 && !lost);                   // there
        EXPECT(looks(limit / 2, limit, &lost) == limit / 2 && !lost);
        EXPECT(looks(limit - 1, limit, &lost) == limit - 1 && !lost);
        EXPECT(looks(limit + 1L, limit, &lost) == limit && lost);       // too late
        EXPECT(looks(-1, limit, &lost) == limit && lost);               // never
    }
    if (!bad) std::printf("ok\n");
    return bad;
}
