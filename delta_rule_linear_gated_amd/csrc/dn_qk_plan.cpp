// dn_qk_plan.cpp -- how a call of the queries' and keys' norms and rotations is split over
// workgroups, and what that needs.  Host code alone.
#include <algorithm>

#include "dn_qk.h"

namespace dn {

constexpr int kQkUnits = 256;   // compute units

// Heads a lane takes, and the workgroups.  More heads a lane share its angles; fewer fill the
// chip.  Measured at 32 + 32 heads of 128, 32768 steps, bf16 (us of calls in a captured graph; rms with
// halves rotated, 4 / 8 / 16 heads): 228 / 220 / 218, backward without weights 299 / 300 / 314.
// As many workgroups as run at once, each walking the token tiles, keep reads and writes apart
// less than a workgroup a tile does: 4 a unit against 8 (backward, l2) 304 -> 348 us (6: 310, 3: 298,
// 2: 341), against one a tile (forward, l2) 210 -> 224, rotation alone 215 -> 221.  But the rotation
// back, whose rows lie head by head on both sides, takes 239 -> 231 (32 + 8 heads, 2 sequences of
// 16384 steps 152 -> 139; but 64 of 512, 32 + 32 heads, 217 -> 283), and with the lengths of a padded
// batch the tiles differ in work (8 sequences of up to 4096 steps, 16 + 16 heads, forward: 101 -> 84):
// then a workgroup a tile, or in the backward, whose workgroups each leave a partial sum, 8 a unit
// (which does not pay with every draw of lengths: this batch, l2, 120 -> 125, 64 sequences of up to 512
// steps 246 -> 287).
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
