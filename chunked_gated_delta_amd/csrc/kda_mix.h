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

// Two values rounded to bf16, to nearest even, in one instruction (a value at a
// time takes one each, and more to pack them), and widened again.
__device__ __forceinline__ uint32_t round2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ float wide_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float wide_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The next bf16 part of x, taken off it: two parts leave an error of at most
// 2^-16 of x, three one of 2^-24.
__device__ __forceinline__ uint32_t cut2(float& a, float& b) {
  const uint32_t u = round2(a, b);
  a -= wide_lo(u);
  b -= wide_hi(u);
  return u;
}
__device__ __forceinline__ uint2 cut_part(float (&x)[4]) {
  const uint32_t a = cut2(x[0], x[1]), b = cut2(x[2], x[3]);
  return make_uint2(a, b);
}
__device__ __forceinline__ uint2 round4(float a, float b, float c, float d) {
  return make_uint2(round2(a, b), round2(c, d));
}

__device__ __forceinline__ void lds_f32x4(const float* src, float* d) {
  const float4 a = *reinterpret_cast<const float4*>(src);
  d[0] = a.x; d[1] = a.y; d[2] = a.z; d[3] = a.w;
}

// Strides of a token array in elements: rows of 16-byte pieces, not negative,
// small enough for 32-bit offsets within 128 rows.
inline bool mix_strides_ok(int64_t token, int64_t head) {
  return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token <= (int64_t)1 << 23 &&
         head <= (int64_t)1 << 23;
}

}  // namespace kda
