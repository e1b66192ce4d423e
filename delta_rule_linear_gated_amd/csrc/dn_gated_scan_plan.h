// dn_gated_scan_plan.h -- which form of the gated linear recurrence a call takes, and what that
// needs (dn_gated_scan_plan.cpp, host code alone); the constants that the kernels share with it.
#pragma once

#include "dn_gated_scan.h"

namespace dn {

constexpr int kGsWaves = 16, kGsRun = 16;         // forward: waves, steps of a run
constexpr int kGsWavesC = 12;                     // forward, chained
constexpr int kGsWavesB = 8;                      // backward: a tile begins at a saved state
constexpr int kGsRunB = kGsSaved / kGsWavesB;
constexpr int kGsUnits = 256, kGsXcds = 8;        // compute units; dies that workgroups go to in turn
static_assert(kGsSaved % kGsRun == 0, "saved states lie at the starts of runs");
constexpr int kGsRange = 0x7fffff00;              // bytes of a buffer range, at most
constexpr int kGsEach = 8;                        // maps that a chained tile's wave gathers
constexpr int kGsHead = 256, kGsMessage = 64 * 8 + 64 * 4;   // bytes of a chain: the counter, a message

struct GsPlan {
    int flat, chain, waves, groups, tiles, reach;   // groups: runs of a channel in a wave (G)
    long strips;
};

long gs_strips(const GsProblem& pr, int groups);
long gs_blocks(long strips, int groups);
GsPlan gs_plan(const GsProblem& pr, bool bwd);
size_t gs_chain_bytes(const GsPlan& p);

struct GsWs {
    size_t states, total;   // the messages lie at the start
};
GsWs gs_ws(const GsProblem& pr, int pass);

}  // namespace dn
