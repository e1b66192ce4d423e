// dn_split.h -- fp32 values as sums of bf16 parts, operands of exact matrix-core products.
#pragma once

#include "dn_device.h"

namespace dn {

// Two floats as two packed bf16; what that leaves of them stays in a, b.  N such steps
// hold 8 N bits of each.  (Written on pairs: one conversion and four more operations a
// step.)
__device__ __forceinline__ unsigned take_bf16(float& a, float& b) {
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    const unsigned u = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{a, b}), bf16x2));
    a -= __builtin_bit_cast(float, u << 16);
    b -= __builtin_bit_cast(float, u & 0xffff0000u);
    return u;
}

}  // namespace dn
