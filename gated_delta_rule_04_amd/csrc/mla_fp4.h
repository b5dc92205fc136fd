// 4-bit latents (gfx950's v_cvt_scalef32 instructions: a code's value times the
// power of two of a float32 scale, a scale byte shifted into its exponent; 255
// gives NaN).  A row's scale bytes from kFp4NaN on stand for NaN: their values
// would leave bf16's range.
#pragma once

#include "mla_launch.h"

namespace mla {

constexpr unsigned kFp4NaN = 253;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// 2 of 8 codes (codes 2i and 2i + 1) as bf16, exactly, and all 8.
template <int I>
__device__ __forceinline__ unsigned fp4_pair(unsigned codes, float scale) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, I));
}
__device__ __forceinline__ u32x4 fp4_values(unsigned codes, float scale) {
  return u32x4{fp4_pair<0>(codes, scale), fp4_pair<1>(codes, scale), fp4_pair<2>(codes, scale),
               fp4_pair<3>(codes, scale)};
}

}  // namespace mla
