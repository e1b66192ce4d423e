// dn_lin_f32_k32.hip -- linear attention's chunk kernel, fp32 I/O, 16 or 32 channels of x and y
#include "dn_linear_kernels.h"

namespace dn {
hipError_t lin_f32_k32(const LinArgs& a, int nv, int mode, hipStream_t s) { return lin_launch<float, 32>(a, nv, mode, s); }
}  // namespace dn
