// q4_stage.cu - keys and values of the prefill route's segments brought from 4 bits to 16.
//
// The tensor-memory prefill kernel reads its K and V tiles by TMA, many times over (once per block
// of query rows), so a long chunk's keys are converted once into a column store of 16-bit values in the
// call's workspace, and the kernel that the bf16 entry uses runs over that.  The values are exact: K in
// bf16, to be multiplied with bf16 queries, and V in fp16, to be multiplied with probabilities that are
// rounded to fp16 as on the other routes (2^-11 of each; with bf16 ones, 2^-8, a 2048-token chunk over 32763
// keys was off by 0.0023 of its norm where the output's own rounding is 0.0017).  Converting inside the kernel instead would repeat the conversion for
// every 256 query rows, on the issue slots that its softmax needs.
//
// Bound by memory: D / 2 + D / 32 bytes read and 2 D written per key and KV head, twice.  A thread
// takes 8 dims (a word of codes, 16 bytes out) of a key and of its value.
#include "packed_stage.cuh"
#include "q4.cuh"

namespace sdpa {

template <int D>
struct Q4Chunk {
  uint32_t kw, vw, kb, vb;
  __device__ __forceinline__ void load(const PackedStore& st, int64_t cell, int c) {
    kw = *reinterpret_cast<const uint32_t*>(st.kc + cell * (D / 2) + 4 * c);
    vw = *reinterpret_cast<const uint32_t*>(st.vc + cell * (D / 2) + 4 * c);
    kb = st.ks[cell * (D / kQ4Group) + c / 4];
    vb = st.vs[cell * (D / kQ4Group) + c / 4];
  }
  __device__ __forceinline__ uint4 keys() const { return q4_words8(kw, kb); }
  __device__ __forceinline__ uint4 values() const { return q4_words8_f16(vw, vb); }
};

template <int D>
__global__ void __launch_bounds__(kPackedStageThreads) sdpa_q4_stage_kernel(PackedStageArgs A) {
  packed_stage<D, Q4Chunk<D>>(A);
}

const void* q4_stage_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q4_stage_kernel<64>;
    case 128: return (const void*)sdpa_q4_stage_kernel<128>;
    default: return (const void*)sdpa_q4_stage_kernel<256>;
  }
}

}  // namespace sdpa
