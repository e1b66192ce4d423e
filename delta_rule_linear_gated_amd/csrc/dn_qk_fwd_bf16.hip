// dn_qk_fwd_bf16.hip -- kernels of dn_qk_kernels.h for bf16 rows, forward.
#include "dn_qk_kernels.h"

namespace dn {
hipError_t qk_fwd_bf16(const QkArgs& a, unsigned blocks, hipStream_t s) { return qk_fwd_type<bf16>(a, blocks, s); }
}  // namespace dn
