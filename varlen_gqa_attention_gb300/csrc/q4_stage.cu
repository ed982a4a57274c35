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
#include "q4.cuh"

namespace sdpa {

// CTA b works on staged column b % pf_cols; its segment is the prefill-route one of that number.
template <int D>
__global__ void __launch_bounds__(kQ4StageThreads) sdpa_q4_stage_kernel(Q4StageArgs A) {
  __shared__ int s_seg;
  const int64_t column = blockIdx.x % A.pf_cols, part = blockIdx.x / A.pf_cols;
  const int64_t parts = gridDim.x / A.pf_cols;
  if (threadIdx.x == 0) s_seg = -1;
  __syncthreads();
  griddep_wait();  // the scheduler's records, and the calls before that used the columns
  griddep_launch();
  for (int s = threadIdx.x; s < A.S; s += blockDim.x)
    if (A.segs[s].route == kRoutePrefill && A.segs[s].pf_col == (int)column) s_seg = s;
  __syncthreads();
  if (s_seg < 0) return;
  const SegRec sg = A.segs[s_seg];
  // the positions the segment's rows see together
  const RowWin w0 = row_window(0, sg.q_len, sg.kv_end, sg.causal, sg.window);
  const int64_t lo = w0.lo, n = (int64_t)sg.kv_end - lo;
  if (n <= 0) return;
  constexpr int W = D / 8;  // words of a row
  const int64_t per_head = n * W, total = per_head * A.Hkv, stride = parts * blockDim.x;
  constexpr int U = 4;
  for (int64_t i0 = part * blockDim.x + threadIdx.x; i0 < total; i0 += U * stride) {
    uint32_t kw[U], vw[U], kb[U], vb[U];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * stride;
      dst[u] = -1;
      if (i < total) {
        const int64_t h = udiv(i, per_head), x = i - h * per_head;
        const int64_t p = lo + x / W;
        const int c = (int)(x % W);
        const int64_t cell = ((int64_t)sg.col * A.Hkv + h) * A.rows + (uint32_t)p % (uint32_t)A.rows;
        kw[u] = *reinterpret_cast<const uint32_t*>(A.st.kc + cell * (D / 2) + 4 * c);
        vw[u] = *reinterpret_cast<const uint32_t*>(A.st.vc + cell * (D / 2) + 4 * c);
        kb[u] = A.st.ks[cell * (D / kQ4Group) + c / 4];
        vb[u] = A.st.vs[cell * (D / kQ4Group) + c / 4];
        dst[u] = (((int64_t)((uint32_t)p % (uint32_t)A.rows_pf) * A.pf_cols + column) * A.Hkv + h) * D + 8 * c;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] < 0) continue;
      *reinterpret_cast<uint4*>(A.k + dst[u]) = q4_words8(kw[u], kb[u]);
      *reinterpret_cast<uint4*>(A.v + dst[u]) = q4_words8_f16(vw[u], vb[u]);
    }
  }
}

const void* q4_stage_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q4_stage_kernel<64>;
    case 128: return (const void*)sdpa_q4_stage_kernel<128>;
    default: return (const void*)sdpa_q4_stage_kernel<256>;
  }
}

}  // namespace sdpa
