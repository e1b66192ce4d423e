// dn_lin_bf16_k32.hip -- linear attention's chunk kernel, bf16 I/O, 16 or 32 channels of x and y
#include "dn_linear_kernels.h"

namespace dn {
hipError_t lin_bf16_k32(const LinArgs& a, int nv, int mode, hipStream_t s) { return lin_launch<bf16, 32>(a, nv, mode, s); }
}  // namespace dn
