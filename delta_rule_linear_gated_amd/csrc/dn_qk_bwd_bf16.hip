// dn_qk_bwd_bf16.hip -- kernels of dn_qk_kernels.h for bf16 rows, backward.
#include "dn_qk_kernels.h"

namespace dn {
hipError_t qk_bwd_bf16(const QkArgs& a, unsigned blocks, hipStream_t s) { return qk_bwd_type<bf16>(a, blocks, s); }
}  // namespace dn
