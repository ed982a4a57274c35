// q4.cuh - the 4-bit column store: its format and the conversions the kernels share.
//
// A store of K (and one of V) is two byte arrays: codes [cols, Hkv, rows, D / 2], where byte i of
// a row holds dim 2i in its low nibble and dim 2i + 1 in its high one, and scales
// [cols, Hkv, rows, D / 32], one byte per 32 dims.  A nibble c under scale byte b stands for
//     (c - 8) * s(b),   s(b) = 2^((b >> 3) - 21) * (1 + (b & 7) / 8).
// c - 8 has at most 4 significant bits and s(b) has 4, so every value has at most 8: it is exact
// in bf16 and (s(b) >= 2^-21 being a multiple of 2^-24, 8 s(b) <= 15360) in fp16 too.  The
// attention kernels therefore see the stored values without a rounding, whichever of the two
// types they multiply in.  Every byte pattern stands for a finite number.
// One KV head's rows of one column are contiguous (the bf16 store interleaves columns and heads
// within a row: at 4 bits that would leave pieces of 32 to 128 bytes per row).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sdpa {

constexpr int kQ4RowAlign = 16;  // store rows are a multiple of this, so that 16 rows of codes and
                                 // of scales are whole 16-byte blocks at every head dim

// s(b) and twice it, as fp32.
__device__ __forceinline__ float q4_scale(uint32_t b) { return __uint_as_float((b << 20) + (106u << 23)); }
__device__ __forceinline__ float q4_scale2(uint32_t b) { return __uint_as_float((b << 20) + (107u << 23)); }

// The scale byte of a group whose largest magnitude is amax: the scale nearest to a seventh of it (ties
// to the even byte), so that |x| / s <= 7 * 17/16 < 7.5 and no code is off by more than half a step.
// The seventh is the fp32 product with 1 / 7: it decides groups within 2^-23 of a border, and is part
// of the format's definition.
// Magnitudes beyond 7 * 1920 take the largest scale and saturate; those below 7 * 2^-21 take byte 0, whose
// half step is 2^-22.
__device__ __forceinline__ uint32_t q4_scale_byte(float amax) {
  const uint32_t u = __float_as_uint(__fmul_rn(amax, 1.f / 7.f));
  const int32_t r = (int32_t)((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (106 << 3);
  return (uint32_t)min(max(r, 0), 255);
}
// (w & mask) | bits in one instruction: the compiler splits it in two when both are constants, so
// `bits` comes in a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(r) : "r"(w), "n"(MASK), "r"(bits));
  return r;
}
// A constant that the compiler keeps in a register.
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// Two bf16 values from nibbles i and i + 4 of a word (shifted so that they are bits 0-3 and 16-19):
// 0x4300 | c is 128 + c, and (128 + c) s - 136 s = (c - 8) s.  136 s = 8 * 17 * (8 to 15) eighths
// has at most 8 significant bits (17 * 15 = 255), so the addend, and with it the result, is exact.
constexpr uint32_t kQ4Bf16 = 0x43004300u;
__device__ __forceinline__ uint32_t q4_pair_bf16(uint32_t w, uint32_t bits, __nv_bfloat162 s2, __nv_bfloat162 z2) {
  const uint32_t x = and_or<0x000F000Fu>(w, bits);  // bits: kQ4Bf16
  const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), s2, z2);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// (s, s) and (-136 s, -136 s) of scale byte b: s is b << 4 above the exponent offset, twice.
__device__ __forceinline__ void q4_scales_bf16(uint32_t b, __nv_bfloat162* s2, __nv_bfloat162* z2) {
  const uint32_t u = b * 0x00100010u + 0x35003500u;
  *s2 = *reinterpret_cast<const __nv_bfloat162*>(&u);
  *z2 = __hmul2(*s2, __float2bfloat162_rn(-136.f));
}

// Two fp16 values from nibbles shifted to bits 6-9 and 22-25: 0x4800 | c << 6 is 8 + c / 2, and
// (8 + c / 2) 2s - 24 s = (c - 8) s; 24 s <= 46080 has 5 significant bits.
constexpr uint32_t kQ4F16 = 0x48004800u;
__device__ __forceinline__ uint32_t q4_pair_f16(uint32_t w, uint32_t bits, __half2 s2, __half2 z2) {
  const uint32_t x = and_or<0x03C003C0u>(w, bits);  // bits: kQ4F16
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&x), s2, z2);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// (2 s(a), 2 s(b)) and (-24 s(a), -24 s(b)).
__device__ __forceinline__ void q4_scales_f16(uint32_t a, uint32_t b, __half2* s2, __half2* z2) {
  *s2 = __floats2half2_rn(q4_scale2(a), q4_scale2(b));
  *z2 = __hmul2(*s2, __float2half2_rn(-12.f));
}

// Pairs of nibbles i and i + 4 of a word, in dim order.
__device__ __forceinline__ uint4 q4_in_order(const uint32_t (&x)[4]) {
  return make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                    __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
}
// The 8 values of one word of codes, in dim order, as bf16 and as fp16.
__device__ __forceinline__ uint4 q4_words8(uint32_t w, uint32_t scale_byte) {
  __nv_bfloat162 s2, z2;
  q4_scales_bf16(scale_byte, &s2, &z2);
  const uint32_t x[4] = {q4_pair_bf16(w, kQ4Bf16, s2, z2), q4_pair_bf16(w >> 4, kQ4Bf16, s2, z2),
                         q4_pair_bf16(w >> 8, kQ4Bf16, s2, z2), q4_pair_bf16(w >> 12, kQ4Bf16, s2, z2)};
  return q4_in_order(x);
}
__device__ __forceinline__ uint4 q4_words8_f16(uint32_t w, uint32_t scale_byte) {
  __half2 s2, z2;
  q4_scales_f16(scale_byte, scale_byte, &s2, &z2);
  const uint32_t x[4] = {q4_pair_f16(w << 6, kQ4F16, s2, z2), q4_pair_f16(w << 2, kQ4F16, s2, z2),
                         q4_pair_f16(w >> 2, kQ4F16, s2, z2), q4_pair_f16(w >> 6, kQ4F16, s2, z2)};
  return q4_in_order(x);
}

// 8 dims of a query row (16 bytes) as the operand words of two k-steps: the conversion of K pairs
// nibbles i and i + 4 of a word, so the fragments pair dims i and i + 4.
__device__ __forceinline__ uint4 q4_q_order(const uint4& a) {
  return make_uint4(__byte_perm(a.x, a.z, 0x5410), __byte_perm(a.x, a.z, 0x7632),
                    __byte_perm(a.y, a.w, 0x5410), __byte_perm(a.y, a.w, 0x7632));
}


// 16-byte blocks from global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Device pointers of a 4-bit store.
struct Q4Store {
  uint8_t* kc;
  uint8_t* ks;
  uint8_t* vc;
  uint8_t* vs;
};

// Pointers present and aligned, rows a multiple of kQ4RowAlign (api.cu).
sdpa_status check_q4_store(const Q4Store& q4, int64_t rows);

struct Q4AttnArgs {
  AttnArgs a;  // k, v unused
  Q4Store st;
  int choice;  // both split-K kernels are launched, and the schedule is one's (hdr->sk_rows)
};

// A call without a schedule (q4_attn.cu): at most kQ4DirectSegs segments, at most kSplitkRows heads a KV head.
constexpr int kQ4DirectSegs = 512;
struct Q4DirectArgs {
  Q4AttnArgs q4;
  const int32_t* seq_info;
  const int32_t* seg_mode;  // NULL, or [S, 2] (causal, window)
  int S;
};

// The keys and values of the prefill route's segments, brought to bf16 and fp16 for the tensor-memory kernel:
// position p of the segment with staged column c goes to row p % rows_pf of column c of a 16-bit
// column store [rows_pf, pf_cols, Hkv, D] (q4_stage.cu).
struct Q4StageArgs {
  const SegRec* segs;  // the scheduler's records
  int S, Hkv, D, pf_cols;
  int64_t rows, rows_pf;
  Q4Store st;
  __nv_bfloat16* k;
  __half* v;
};
constexpr int kQ4StageThreads = 256;
const void* q4_stage_kernel_ptr(int D);

// Entry points (q4_attn.cu).
constexpr int kQ4Threads = 160;  // four warps of attention, one that loads
// The tensor-memory kernel for segments of several rows (q4_tile.cu; D = 64, 128): one CTA per SM, units of
// kQ4TileRows packed rows, tiles of kQ4TileKeys keys.
constexpr int kQ4TileRows = 128;
constexpr int kQ4TileKeys = 128;
constexpr int kQ4TileThreads = 576;
const void* q4_tile_kernel_ptr(int D);
int q4_tile_smem_bytes(int D);
const void* q4_splitk_kernel_ptr(int D);
const void* q4_direct_kernel_ptr(int D);
int q4_splitk_smem_bytes(int D);

}  // namespace sdpa
