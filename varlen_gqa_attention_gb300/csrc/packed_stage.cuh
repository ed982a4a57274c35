// packed_stage.cuh - keys and values of the prefill route's segments brought from a store of codes to a column store
// of 16-bit values in the workspace (q4_stage.cu, q8_stage.cu).
#pragma once

#include "packed.cuh"

namespace sdpa {

// CTA b works on staged column b % pf_cols; its segment is the prefill-route one of that number.
// F: a chunk of 8 dims of a key and its value as stored (load), and as 16-bit values (keys, values).
template <int D, typename F>
__device__ __forceinline__ void packed_stage(const PackedStageArgs& A) {
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
  constexpr int W = D / 8;  // chunks of a row
  const int64_t per_head = n * W, total = per_head * A.Hkv, stride = parts * blockDim.x;
  constexpr int U = 4;
  for (int64_t i0 = part * blockDim.x + threadIdx.x; i0 < total; i0 += U * stride) {
    F x[U];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * stride;
      dst[u] = -1;
      if (i < total) {
        const int64_t h = udiv(i, per_head), j = i - h * per_head;
        const int64_t p = lo + j / W;
        const int c = (int)(j % W);
        const int64_t cell = ((int64_t)sg.col * A.Hkv + h) * A.rows + (uint32_t)p % (uint32_t)A.rows;
        x[u].load(A.st, cell, c);
        dst[u] = (((int64_t)((uint32_t)p % (uint32_t)A.rows_pf) * A.pf_cols + column) * A.Hkv + h) * D + 8 * c;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] < 0) continue;
      *reinterpret_cast<uint4*>(A.k + dst[u]) = x[u].keys();
      *reinterpret_cast<uint4*>(A.v + dst[u]) = x[u].values();
    }
  }
}

}  // namespace sdpa
