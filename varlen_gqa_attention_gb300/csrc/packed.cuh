// packed.cuh - what the 4-bit and the 8-bit column store have in common.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sdpa {

// Store rows are a multiple of this: at 4 bits 16 rows of codes and of scales are whole 16-byte blocks at every
// head dim, at 8 bits 16 rows of a head share a scale.
constexpr int kPackedRows = 16;

// The blocks of kPackedRows store rows that a segment (q_len > 0, kv_end) writes to: `count` of them from `first` on, on a
// ring of all of a column's blocks (count may be one more than those).
struct BlockRun {
  int64_t first, count;
};
__host__ __device__ inline BlockRun block_run(int32_t q_len, int32_t kv_end) {
  if (kv_end <= 0) return {0, 0};  // no position: nothing is written
  const int64_t first = (kv_end > q_len ? kv_end - q_len : 0) / kPackedRows;
  return {first, (kv_end - 1) / kPackedRows - first + 1};
}
// Whether two runs share a block of a ring of `ring`.
__host__ __device__ inline bool runs_meet(const BlockRun& a, const BlockRun& b, int64_t ring) {
  if (a.count == 0 || b.count == 0) return false;
  const int64_t d = ((b.first - a.first) % ring + ring) % ring;  // where b's begins, counted from a's
  return d < a.count || d + b.count > ring;
}
// Whether two segments of one column write to one block.
__host__ __device__ inline bool blocks_meet(int32_t a_len, int32_t a_end, int32_t b_len, int32_t b_end, int64_t rows) {
  return runs_meet(block_run(a_len, a_end), block_run(b_len, b_end), rows / kPackedRows);
}

// Device pointers of a store of codes and scales.
struct PackedStore {
  uint8_t* kc;
  uint8_t* ks;
  uint8_t* vc;
  uint8_t* vs;
};

// Pointers present and aligned, rows a multiple of kPackedRows; `bits` 4 or 8 (api.cu).
sdpa_status check_packed_store(const PackedStore& st, int bits, int64_t rows);

constexpr int kPackedThreads = 160;  // of the kernels for few rows: four warps of attention, one that loads
// A call without a schedule (packed_attn.cuh): at most kPackedDirectSegs segments, at most kSplitkRows heads a KV
// head.
constexpr int kPackedDirectSegs = 512;
template <class Args>
struct PackedDirectArgs {
  Args packed;
  const int32_t* seq_info;
  const int32_t* seg_mode;  // NULL, or [S, 2] (causal, window)
  int S;
};

// The keys and values of the prefill route's segments, brought to bf16 and fp16 for the tensor-memory kernel:
// position p of the segment with staged column c goes to row p % rows_pf of column c of a 16-bit
// column store [rows_pf, pf_cols, Hkv, D] (q4_stage.cu, q8_stage.cu).
struct PackedStageArgs {
  const SegRec* segs;  // the scheduler's records
  int S, Hkv, D, pf_cols;
  int64_t rows, rows_pf;
  PackedStore st;
  __nv_bfloat16* k;
  __half* v;
};
constexpr int kPackedStageThreads = 256;

// The tensor-memory kernel for segments of several rows (packed_tile.cuh; D = 64, 128): one CTA per SM, units of
// kPackedTileRows packed rows, tiles of kPackedTileKeys keys.
constexpr int kPackedTileRows = 128;
constexpr int kPackedTileKeys = 128;
constexpr int kPackedTileThreads = 576;

// A constant that the compiler keeps in a register.
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}

// 16-byte blocks from global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace sdpa
