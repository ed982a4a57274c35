// packed.cuh - what the 4-bit and the 8-bit column store have in common.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sdpa {

// Store rows are a multiple of this: at 4 bits 16 rows of codes and of scales are whole 16-byte blocks at every
// head dim, at 8 bits 16 rows of a head share a scale.
constexpr int kPackedRows = 16;

// Whether two segments (q_start, q_len, col, kv_end) of one column, q_len > 0, write to one block of kPackedRows store
// rows.  Each writes a run of blocks, on a ring of all the column's blocks.
__host__ __device__ inline bool blocks_meet(int32_t a_len, int32_t a_end, int32_t b_len, int32_t b_end, int64_t rows) {
  if (a_end <= 0 || b_end <= 0) return false;  // no position: nothing is written
  const int64_t ring = rows / kPackedRows;
  const int64_t a0 = (a_end > a_len ? a_end - a_len : 0) / kPackedRows, an = (a_end - 1) / kPackedRows - a0 + 1;
  const int64_t b0 = (b_end > b_len ? b_end - b_len : 0) / kPackedRows, bn = (b_end - 1) / kPackedRows - b0 + 1;
  const int64_t d = ((b0 - a0) % ring + ring) % ring;  // where b's run begins, counted from a's
  return d < an || d + bn > ring;
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
