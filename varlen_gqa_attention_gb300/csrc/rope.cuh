// rope.cuh - arguments and entry points of the rotary and step kernels (rope.cu).
#pragma once

#include "q4.cuh"

namespace sdpa {

constexpr int kRopeAxes = 4;       // position axes at most
constexpr int kRopeThreads = 256;
constexpr int kStepRows = 16;      // packed rows of one CTA at most

// The rotation: pair j of a row belongs to the axis whose section [sec_end[a - 1], sec_end[a])
// holds it (sec_end of axes that are not there: INT_MAX).
struct RopeArgs {
  const float2* table;  // [P, half] (cos, sin)
  int64_t P;
  int half, axes;
  int sec_end[kRopeAxes];
  const int32_t* pos;   // [axes, T], or null: the row's position in its sequence
  int64_t pos_stride;
  int inverse;
};

struct RopeRowsArgs {
  RopeArgs r;
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t x_rs, x_hs, o_rs, o_hs, T;
  int H, parts;  // parts: warps that share a row
  int32_t* status_dev;
};

// A step's rows and the store they belong to.
struct StepArgs {
  RopeArgs r;
  const int32_t* seq_info;
  const int32_t* seg_mode;  // NULL, or [S, 2] (causal, window)
  int S, window, cols, Hq, Hkv;
  int cr;                   // read-back: packed rows per CTA
  int per;                  // append: passes per CTA
  int64_t T, rows;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs;
  __nv_bfloat16 *q_out, *k_out, *v_out;  // k_out, v_out: rows read back
  int64_t o_rs, o_hs;
  __nv_bfloat16 *k_store, *v_store;
  Q4Store q4;
  int32_t* status_dev;
};

const void* rope_kernel_ptr(int D, bool interleaved);
const void* rope_append_kernel_ptr(int D, bool interleaved, bool q4);
const void* q4_unpack_kernel_ptr(int D);
int rope_heads_per_pass(int D);  // heads of one row that a warp takes at a time

}  // namespace sdpa
