// 4-bit latents (gfx950's v_cvt_scalef32 instructions: a code's value times the
// power of two of a float32 scale, a scale byte shifted into its exponent; 255
// gives NaN).
#pragma once

#include "mla_launch.h"

namespace mla {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// 8 codes as 8 bf16, exactly.
__device__ __forceinline__ u32x4 fp4_values(unsigned codes, float scale) {
  return u32x4{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
               __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3))};
}

}  // namespace mla
