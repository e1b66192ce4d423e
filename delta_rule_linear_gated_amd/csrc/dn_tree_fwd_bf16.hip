// dn_tree_fwd_bf16.hip -- nodes of a drafted-token tree, bf16 I/O
#include "dn_tree_kernels.h"

namespace dn {
hipError_t tree_fwd_bf16(const TreeArgs& a, hipStream_t s) { return tree_launch<bf16>(a, s); }
}  // namespace dn
