// dn_qk_fwd_f32.hip -- kernels of dn_qk_kernels.h for fp32 rows, forward.
#include "dn_qk_kernels.h"

namespace dn {
hipError_t qk_fwd_f32(const QkArgs& a, unsigned blocks, hipStream_t s) { return qk_fwd_type<float>(a, blocks, s); }
}  // namespace dn
