// dn_tree_fwd_f32.hip -- nodes of a drafted-token tree, fp32 I/O
#include "dn_tree_kernels.h"

namespace dn {
hipError_t tree_fwd_f32(const TreeArgs& a, hipStream_t s) { return tree_launch<float>(a, s); }
}  // namespace dn
