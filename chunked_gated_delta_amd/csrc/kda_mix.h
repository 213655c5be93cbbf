// Shared pieces of the token mixers beside the KDA core (linear attention with
// a decay for each head, causal attention): 16-bit MFMA operands from LDS, and
// the exact splits of fp32 values into bf16 parts.  Internal header.
#pragma once

#include "kda_common.h"
#include "kda_host.h"
#include "kda_token.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Transposing LDS read: a group of 16 lanes reads 4 rows of 16 elements, lane l
// the 4 elements from column 4 (l % 4) of row l / 4 at its own address, and
// lane l gets column l % 16, rows 0..3.
__device__ __forceinline__ uint2 tr_read(const uint16_t* p) {
  typedef __attribute__((address_space(3))) s16x4* lds_t;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(void*)p));
}
__device__ __forceinline__ bf16x8 join(uint2 a, uint2 b) {
  return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}

// The next bf16 part of x, taken off it: two parts leave an error of at most
// 2^-16 of x, three one of 2^-24.
__device__ __forceinline__ bf16x4 cut_part(float (&x)[4]) {
  bf16x4 p;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    p[r] = (__bf16)x[r];
    x[r] -= (float)p[r];
  }
  return p;
}

// Strides of a token array in elements: rows of 16-byte pieces, not negative,
// small enough for 32-bit offsets within 128 rows.
inline bool mix_strides_ok(int64_t token, int64_t head) {
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token <= (int64_t)1 << 23 &&
         head <= (int64_t)1 << 23;
}

}  // namespace kda
