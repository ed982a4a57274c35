// q8_stage.cu - keys and values of the prefill route's segments brought from 8 bits to 16, as q4_stage.cu does from 4:
// exactly, K to bf16 and V / 16 to fp16 (V itself can be -65536, which fp16 does not hold); the prefill kernels multiply
// their output by the 16 again.
//
// Bound by memory: D and an eighth of a byte read and 2 D written per key and KV head, twice.  24001 keys of 2 heads,
// D = 128: 11 us (4-bit: 13 for 32763).
#include "packed_stage.cuh"
#include "q8.cuh"

namespace sdpa {

template <int D>
struct Q8Chunk {
  uint2 kw, vw;
  uint32_t kb, vb;
  __device__ __forceinline__ void load(const PackedStore& st, int64_t cell, int c) {
    kw = *reinterpret_cast<const uint2*>(st.kc + cell * D + 8 * c);
    vw = *reinterpret_cast<const uint2*>(st.vc + cell * D + 8 * c);
    kb = st.ks[cell / kPackedRows];
    vb = st.vs[cell / kPackedRows];
  }
  __device__ __forceinline__ uint4 keys() const {
    const __nv_bfloat162 s = q8_scale_bf16(kb);
    const uint2 a = q8_words4(kw.x, s), b = q8_words4(kw.y, s);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ uint4 values() const {
    const uint32_t w = q8_scale_f16x2(vb);
    const __half2 t = *reinterpret_cast<const __half2*>(&w), z = __hmul2(t, __float2half2_rn(-1152.f));
    return make_uint4(q8_pair_f16<false>(vw.x, kQ8Magic, t, z), q8_pair_f16<true>(vw.x, kQ8Magic, t, z),
                      q8_pair_f16<false>(vw.y, kQ8Magic, t, z), q8_pair_f16<true>(vw.y, kQ8Magic, t, z));
  }
};

template <int D>
__global__ void __launch_bounds__(kPackedStageThreads) sdpa_q8_stage_kernel(PackedStageArgs A) {
  packed_stage<D, Q8Chunk<D>>(A);
}

const void* q8_stage_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q8_stage_kernel<64>;
    case 128: return (const void*)sdpa_q8_stage_kernel<128>;
    default: return (const void*)sdpa_q8_stage_kernel<256>;
  }
}

}  // namespace sdpa
