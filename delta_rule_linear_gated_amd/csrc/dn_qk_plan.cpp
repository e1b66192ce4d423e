// dn_qk_plan.cpp -- how a call of the queries' and keys' norms and rotations is split over
// workgroups, and what that needs.  Host code alone.
#include <algorithm>

#include "dn_qk.h"

namespace dn {

constexpr int kQkUnits = 256;   // compute units

// Heads a lane takes, and the workgroups.  More heads a lane share its angles; fewer fill the
// chip.  Measured at 32 + 32 heads of 128, 32768 steps, bf16 (us, rms with halves rotated, 4 / 8 /
// 16 heads): 234 / 223 / 217, backward without weights 347 / 329 / 328, with few tokens (16 + 16
// heads, 1024 steps) 7.5 / 8.0 / 7.3.
// As many workgroups as run at once, each walking the token tiles, keep reads and writes apart
// less than a workgroup a tile does: 4 a unit against 8 (backward, l2) 305 -> 350 us (6: 311, 3: 299,
// 2: 343), against one a tile (forward, l2) 211 -> 220, rotation alone 212 -> 221.  But the rotation
// back, whose rows lie head by head on both sides, takes 231 -> 217, and with the lengths of a
// padded batch the tiles differ in work (8 sequences of up to 4096 steps, 16 + 16 heads, forward:
// 101 -> 85): then a workgroup a tile, or in the backward, whose workgroups each leave a partial
// sum, 8 a unit.
void qk_split(QkArgs* a, bool bwd) {
    const long tokens = (long)a->B * a->T, per_wg = 256 / (a->d / 8);
    const long tiles = (tokens + per_wg - 1) / per_wg;
    const long most = std::max(a->side[0].heads, a->side[1].heads);   // heads may be any int: sums of them are not
    int per = 8;
    auto groups = [&](int side) { return ((long)a->side[side].heads + per - 1) / per; };
    while (per > 1 && (per >= 2 * most || tiles * (groups(0) + groups(1)) < 4 * kQkUnits)) per /= 2;
    a->per = per;
    a->groups[0] = (int)groups(0);
    a->groups[1] = (int)groups(1);
    const long all = std::max(groups(0) + groups(1), 1L);
    const bool uneven = a->lens || a->back;
    a->tiles = (int)(uneven && !bwd ? tiles : std::min<long>(tiles, std::max((uneven ? 8 : 4) * kQkUnits / all, 1L)));
}

bool qk_fits(const QkArgs& in) {
    QkArgs a = in;
    a.back = 1;   // the most workgroups
    qk_split(&a, false);
    return (long)a.tiles * ((long)a.groups[0] + a.groups[1]) < (1L << 32) / 256;
}

size_t qk_workspace_bytes(const QkArgs& in) {
    QkArgs a = in;
    if ((long)a.B * a.T == 0) return 0;
    a.back = 1;   // the most workgroups, as with lengths
    qk_split(&a, true);
    return (size_t)a.tiles * ((size_t)a.groups[0] + a.groups[1]) * a.d * 4;
}

}  // namespace dn
