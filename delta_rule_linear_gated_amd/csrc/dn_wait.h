// dn_wait.h -- a wait, with an end, for what another workgroup of the same launch writes.
#pragma once

#include <hip/hip_runtime.h>

namespace dn {

// Looks until `there`; after `looks` (1 at least) of them gives up, which has to make `there` true.
template <typename There, typename Look, typename GiveUp>
__host__ __device__ inline void wait_until(There there, Look look, GiveUp give_up, int looks) {
    for (int left = looks; !there();) {
        look();
        if (--left == 0) give_up();
    }
}

}  // namespace dn
