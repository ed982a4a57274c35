// q8.cuh - the 8-bit column store: its format and the conversions the kernels share.
//
// A store of K (and one of V) is two byte arrays: codes [cols, Hkv, rows, D] and scales [cols, Hkv, rows / 16],
// one byte for each block of 16 rows of a head.  A code c under scale byte b stands for
//     (c - 128) * s(b),   s(b) = 2^(min(b, 29) - 20).
// c - 128 has at most 8 significant bits, so every value is exact in bf16 and, being a multiple of 2^-20 of at
// most 128 * 2^9, all but -65536 (which no append writes) is exact in fp16 too.  Every byte pattern stands for a
// finite number, so that a row that holds no position cannot spoil a product whose other factor is 0.
// The scales are powers of two so that a block may be coded again as rows come to it: under a smaller scale that
// is exact, and under a larger one it is one rounding by half a step, which adds up over all growths of a block
// to less than one step of its last scale.
// (Codes and not 8-bit floating-point numbers: normal values are off by a third as much, and no code is a NaN.)
#pragma once

#include <cfloat>

#include <cuda.h>

#include "packed.cuh"

namespace sdpa {

constexpr int kQ8Bias = 20, kQ8Top = 29;

// s(b) as fp32.
__device__ __forceinline__ float q8_scale(uint32_t b) {
  return __uint_as_float((min(b, (uint32_t)kQ8Top) + (127 - kQ8Bias)) << 23);
}
// The scale byte of a block whose largest magnitude is amax: that of the smallest scale with amax <= 127 s.
// 127 = 1.984375 * 2^6, so the exponent of s is amax's less 6, or less 5 where the fraction is beyond 0x7E0000.
__device__ __forceinline__ uint32_t q8_scale_byte(float amax) {
  const int32_t b = (int32_t)((__float_as_uint(amax) + 0x1FFFFu) >> 23) - (127 + 6 - kQ8Bias);
  return (uint32_t)min(max(b, 0), kQ8Top);
}

// Two bf16 values (c - 128) from bytes 0 and 2 of x: 0x4300 | (c & 127) is 128 + (c & 127), and 0x4300 or 0x4380,
// by the code's top bit, is 128 or 256; the difference is exact.
__device__ __forceinline__ __nv_bfloat162 q8_pair_bf16(uint32_t x) {
  const uint32_t a = (x & 0x007F007Fu) | 0x43004300u, z = (~x & 0x00800080u) | 0x43004300u;
  return __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&z));
}
// The four values of a word of codes under scale s, as bf16 in dim order.
__device__ __forceinline__ uint2 q8_words4(uint32_t w, __nv_bfloat162 s2) {
  const __nv_bfloat162 lo = __hmul2(q8_pair_bf16(__byte_perm(w, 0, 0x4140)), s2);
  const __nv_bfloat162 hi = __hmul2(q8_pair_bf16(__byte_perm(w, 0, 0x4342)), s2);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
__device__ __forceinline__ __nv_bfloat162 q8_scale_bf16(uint32_t b) { return __float2bfloat162_rn(q8_scale(b)); }

struct Q8AttnArgs {
  CUtensorMap k, v;  // the store's codes as [cols * Hkv, rows, D] bytes, in boxes of 16 rows (api.cu)
  AttnArgs a;        // k, v unused
  PackedStore st;
  int choice;  // both split-K kernels are launched, and the schedule is one's (hdr->sk_rows)
};

const void* q8_splitk_kernel_ptr(int D);
const void* q8_direct_kernel_ptr(int D);
int q8_splitk_smem_bytes(int D);
const void* q8_stage_kernel_ptr(int D);

}  // namespace sdpa
