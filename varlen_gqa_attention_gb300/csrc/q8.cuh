// q8.cuh - the 8-bit column store: its format and the conversions the kernels share.
//
// A store of K (and one of V) is two byte arrays: codes [cols, Hkv, rows, D] and scales [cols, Hkv, rows / 16],
// one byte for each block of 16 rows of a head.  A code c under scale byte b stands for
//     (c - 128) * s(b),   s(b) = 2^(min(b, 29) - 20).
// c - 128 has at most 8 significant bits, so every value is exact in bf16 and, being a multiple of 2^-20 of at
// most 128 * 2^9, a sixteenth of it is exact in fp16.  Every byte pattern stands for a finite number, so that a row
// that holds no position cannot spoil a product whose other factor is 0.
// The scales are powers of two so that a block may be coded again as rows come to it: under a smaller scale that
// is exact, and under a larger one it is one rounding by half a step, which adds up over all growths of a block
// to less than one step of the largest scale it has had.
// (Codes and not 8-bit floating-point numbers: normal values are off by 0.011 of their deviation, root mean square at
// D = 128, where e4m3 numbers are by 0.027, and no code is a NaN.)
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

// What the attention kernels multiply: values / 16 in fp16, exact, which one fused multiply-add makes of a code.
// 0x6400 | c is 1024 + c, and (1024 + c) t - 1152 t = (c - 128) t with t = s / 16, whose largest addend is
// 1152 * 2^5; every term and the result are exact.
constexpr uint32_t kQ8Magic = 0x64646464u;  // the high byte of 1024 in fp16, four times
// (t, t) of a scale byte: 2^(b - 24) in fp16, below 2^-14 a subnormal number.
__device__ __forceinline__ uint32_t q8_scale_f16x2(uint32_t byte) {
  const uint32_t b = min(byte, (uint32_t)kQ8Top);
  const uint32_t t = b < 10 ? 1u << b : (b - 9) << 10;
  return t | t << 16;
}
// Two values / 16 from bytes 0 and 1 (HI: 2 and 3) of x; magic: kQ8Magic in a register, z = -1152 t.
template <bool HI>
__device__ __forceinline__ uint32_t q8_pair_f16(uint32_t x, uint32_t magic, __half2 t, __half2 z) {
  const uint32_t u = __byte_perm(x, magic, HI ? 0x4342 : 0x4140);
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&u), t, z);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Query rows in fp16: a row times 2^(14 - e), e being the exponent of its largest magnitude (but at most 2^126, so
// that rows of less than 2^-112 stay as much below 2^14; a row with an infinity keeps it).  What is above 2^-31
// of the largest magnitude is exact, what is below is off by at most 2^-39 of it.
__device__ __forceinline__ float q8_row_amax(const uint4& w, float amax) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xFFFF0000u))));
  return amax;
}
// The exponent field of the factor.
__device__ __forceinline__ uint32_t q8_row_up(float amax) {
  return 268u - min(max(__float_as_uint(amax) >> 23, 15u), 254u);
}
__device__ __forceinline__ uint4 q8_row_f16(const uint4& w, float mul) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 v = __floats2half2_rn(__uint_as_float(x[k] << 16) * mul, __uint_as_float(x[k] & 0xFFFF0000u) * mul);
    f[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(f[0], f[1], f[2], f[3]);
}
// The scale of such a row's scores against keys / 16: finite and not 0, so that a masked score stays -infinity and
// a score of 0 stays 0.
__device__ __forceinline__ float q8_row_scale(uint32_t up, float scale_log2) {
  return fminf(fmaxf(16.f * scale_log2 * __uint_as_float((254u - up) << 23), FLT_MIN), FLT_MAX);
}

// The store's codes as [cols * Hkv, rows, D] bytes for TMA, in boxes of 16 rows and of q8_box_rows (api.cu).  (A
// warp's copies go out one after another: the 16 small boxes of a stage of 128 keys took 0.5 us, which one
// sequence's CTAs waited for.)
constexpr int q8_box_rows(int D) { return D == 256 ? 64 : 128; }
struct Q8AttnArgs {
  CUtensorMap k, v, k_box, v_box;
  AttnArgs a;        // k, v unused
  PackedStore st;
  int choice;  // both split-K kernels are launched, and the schedule is one's (hdr->sk_rows)
};

const void* q8_splitk_kernel_ptr(int D);
const void* q8_direct_kernel_ptr(int D);
int q8_splitk_smem_bytes(int D);
const void* q8_stage_kernel_ptr(int D);
constexpr float kQ8StagedMul = 16.f;  // a staged value stands for this many times itself
const void* q8_tile_kernel_ptr(int D);
int q8_tile_smem_bytes(int D);

}  // namespace sdpa
