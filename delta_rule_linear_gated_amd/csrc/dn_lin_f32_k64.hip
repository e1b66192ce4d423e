// dn_lin_f32_k64.hip -- linear attention's chunk kernel, fp32 I/O, 64 channels of x and y
#include "dn_linear_kernels.h"

namespace dn {
hipError_t lin_f32_k64(const LinArgs& a, int nv, int mode, hipStream_t s) { return lin_launch<float, 64>(a, nv, mode, s); }
}  // namespace dn
