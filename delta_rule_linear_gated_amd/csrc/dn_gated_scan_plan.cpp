// dn_gated_scan_plan.cpp -- the gated linear recurrence's forms: strips, tiles, waves, whether
// chained, and the bytes of workspaces and saved states.  Host code alone.
#include "dn_gated_scan_plan.h"

#include <algorithm>

namespace dn {

namespace {

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// Strips of 64 / G channels: of one head's row, or (flat) of the channels of all heads in a row, so
// that odd widths leave no lane idle, but lanes of two heads read twice the cache lines.  Measured
// (us, forward / backward, one head's -> flat):
//     marching, 280 heads, 2000 steps     d 67 (47 % of the lanes idle) 141 / 218 -> 101 / 180, d 100 (22 %) 151 / 257 -> 153 / 277
//     marching, 300 heads of 100, 3334 steps      258 / 466 -> 275 / 498
//     chained, 80 heads of 100, 3334 steps        75 / 127 -> 72 / 128, fp32 88 / 160 -> 88 / 165
//     one tile, fp32, 777 steps                   15 heads of 67 8.1 / 11.6 -> 10.6 / 15.5, 150 heads of 24 11.1 / 18.8 -> 11.2 / 17.3
// So flat where more than a quarter of the lanes would idle, in every form, or where several runs a
// wave would take more than one round of the chip; never where a strip's rows lie further apart
// than a 31-bit byte offset.
bool gs_flat(const GsProblem& pr, int groups) {
    const long C = 64 / groups, per = (pr.d + C - 1) / C, rows = 63 / pr.d + 2;   // a strip touches at most that many
    if (rows * pr.T >= kGsRange / 4 / pr.d) return false;
    return groups > 1 ? (long)pr.B * pr.H * per > kGsUnits : 4 * pr.d < 3 * per * C;
}

}  // namespace

long gs_strips(const GsProblem& pr, int groups) {
    const long BH = (long)pr.B * pr.H, C = 64 / groups;
    return gs_flat(pr, groups) ? (BH * pr.d + C - 1) / C : BH * ((pr.d + C - 1) / C);
}
long gs_blocks(long strips, int groups) {   // G > 1: a whole number of 64-channel groups for every XCD
    const long all = groups > 1 ? kGsXcds * groups : 1;
    return (strips + all - 1) / all * all;
}
// Which form.  Measured (us, forward / backward, bf16, coupled; marching with the best G -> chained):
//     64 strips, 8192 steps        77 / 132 -> 74 / 113      4 strips, 4096 steps          18.5 / 26.5 -> 14.6 / 15.6
//     157 strips, 4096 steps     109 / 191 -> 93 / 160       15 strips (fp32), 777 steps     6.8 / 9.9 -> 13.0 / 14.4
//     32 strips, 32768 steps     180 / 297 -> 131 / 206      32 strips, 512 steps             6.1 / 8.7 -> 13.2 / 14.7
// (256 strips, 4096 steps, as many bytes as 32 strips, 32768 steps: marching 114 / 200; a copy of as
// many bytes, half of them written, 105 / 183.)
// So: up to 1024 steps march, as many runs of a channel in a wave as make one tile of them and still
// leave one round of workgroups (224 strips, 1000 steps, of one tile -> so: 43 / 92 -> 30 / 46 us), a
// round being two workgroups of a unit forward and one backward.  Forward with one instead: 128
// strips, 300 steps 9.5 -> 10.5, 57 strips (fp32), 777 steps 11.0 -> 13.2, 224 strips, 300 steps 14.3 ->
// 14.8; backward with two: 128 strips, 300 steps 13.9 -> 15.7, 64 strips, 1000 steps 16.3 -> 22, 160
// strips, 600 steps 25.6 -> 30.5.  One bound for all lengths, though with one round 64 strips, 1000
// steps forward would take 12.1 instead of 13.0, 160 strips, 600 steps 18.9 instead of 19.4.  Longer
// ones are chained where marching would leave more than a fifth of the chip idle; else strips of 64
// channels march.
// Waves: up to 128 steps only those whose runs they are (131072 channels, 16 steps, of 16 waves -> of
// one: 46 -> 6.8 us).  Longer, forward: 16 where a unit has one strip (256 strips, 4096 steps:
// 113 us, of 8 waves 117), 8 where it has two, whose loads then overlap (2048 strips, 512 steps:
// 130 -> 111; 512 strips, 4096 steps: 222 -> 217; fp32, 1024 strips: 625 both).
constexpr int kGsShort = 1024;
GsPlan gs_plan(const GsProblem& pr, bool bwd) {
    GsPlan p{};
    p.groups = 1;
    p.strips = gs_strips(pr, 1);
    p.waves = pr.T <= 16 ? 1 : pr.T <= 64 ? 4 : bwd || pr.T <= 128 || p.strips >= 2 * kGsUnits ? 8 : kGsWaves;
    int tile = 16 * p.waves;
    const long rounds = (p.strips + kGsUnits - 1) / kGsUnits;
    if (pr.T > 128 && pr.T <= kGsShort && p.strips < kGsUnits) {
        auto blocks = [&](int g) { return gs_blocks(gs_strips(pr, g), g); };
        while (128 * p.groups < pr.T && blocks(2 * p.groups) <= (bwd ? 1 : 2) * kGsUnits) p.groups *= 2;
        if (p.groups > 1) p.waves = 8, tile = 128;
        p.strips = gs_strips(pr, p.groups);
    } else if (pr.T > kGsShort && p.strips * 5 < rounds * kGsUnits * 4) {
        const int ctile = bwd ? kGsSaved : kGsWavesC * kGsRun;
        if (p.strips * (((long)pr.T + ctile - 1) / ctile) < (1L << 30)) {
            p.chain = 1;
            tile = ctile;
            // the tiles of a strip that are in flight at once (twice as many: within 2 %), as far as every
            // wave has eight to ask for (more for one strip, 65536 steps: 29 -> 33 us)
            p.reach = (int)std::min<long>((bwd ? kGsWavesB : kGsWavesC) * kGsEach, std::max<long>(4, kGsUnits / p.strips));
        }
    }
    p.flat = gs_flat(pr, p.groups);
    p.tiles = (int)(((long)pr.T + (long)tile * p.groups - 1) / ((long)tile * p.groups));
    return p;
}

size_t gs_chain_bytes(const GsPlan& p) { return p.chain ? kGsHead + (size_t)p.strips * p.tiles * kGsMessage : 0; }

GsWs gs_ws(const GsProblem& pr, int pass) {
    GsWs w{};
    if (pass != 1) w.states = gs_chain_bytes(gs_plan(pr, false));
    if (pass != 0) w.states = std::max(w.states, gs_chain_bytes(gs_plan(pr, true)));
    w.states = al256(w.states);
    w.total = w.states + (pass == 2 ? al256(gs_states_bytes(pr)) : 0);
    return w;
}

size_t gs_states_bytes(const GsProblem& pr) {
    return (size_t)pr.B * pr.H * (((size_t)pr.T + kGsSaved - 1) / kGsSaved) * pr.d * 4;
}
size_t gs_workspace_bytes(const GsProblem& pr, int pass) { return gs_ws(pr, pass).total; }
bool gs_fits(const GsProblem& pr) {
    if (pr.B == 0 || pr.H == 0) return true;
    return (long)pr.B * pr.H <= 0x7fffffffL && gs_strips(pr, 1) < (1L << 32) / (64 * kGsWaves);
}

}  // namespace dn
