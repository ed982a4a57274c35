// rope_api.cu - C entries of the rotary and step kernels: argument checks and launches.
//
// Every check runs before any CUDA call.  The launches are asynchronous, need no workspace and
// allocate nothing, so a call can be captured in a CUDA graph.
#include <algorithm>
#include <climits>
#include <mutex>

#include "rope.cuh"

namespace sdpa {
namespace {

constexpr int kMaxHeads = 1 << 20;  // of one row (the kernels count a CTA's passes over them in 32 bits)

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool bad_strides(int64_t rs, int64_t hs) { return rs < 0 || hs < 0 || rs % 8 || hs % 8; }

// SMs of the current device (asked once per device).
sdpa_status device_sms(int* sms) {
  static std::mutex mu;
  static int known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(SDPA_ERR_CUDA, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    e = cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "SM count: %s", cudaGetErrorString(e));
  }
  *sms = known[dev];
  return SDPA_OK;
}

// Checks a rotation and turns it into the kernels' form.  `own_position`: positions may be NULL.
sdpa_status take_rotation(const sdpa_rotation* r, int64_t T, int D, bool own_position, int inverse, RopeArgs* out) {
  if (!r || !r->table) return fail(SDPA_ERR_NULL, "rotation or its table is NULL");
  if (!aligned16(r->table)) return fail(SDPA_ERR_ALIGN, "the rotation table must be 16-byte aligned");
  if (r->table_rows < 1 || r->table_rows > INT_MAX)
    return fail(SDPA_ERR_SHAPE, "table_rows %lld outside [1, 2^31)", (long long)r->table_rows);
  if (r->rot_dims < 16 || r->rot_dims > D || r->rot_dims % 16)
    return fail(SDPA_ERR_ARG, "rot_dims %d: a multiple of 16, at most the head dim %d", r->rot_dims, D);
  if (r->table_rows * (r->rot_dims / 2) > INT_MAX)
    return fail(SDPA_ERR_SHAPE, "a table of %lld x %d pairs: at most 2^31 - 1", (long long)r->table_rows,
                r->rot_dims / 2);
  if (r->axes < 1 || r->axes > kRopeAxes) return fail(SDPA_ERR_ARG, "%d position axes: 1 to %d", r->axes, kRopeAxes);
  if (!r->positions && T > 0 && !(own_position && r->axes == 1))
    return fail(SDPA_ERR_NULL, "positions is NULL%s", own_position ? " and there are several axes" : "");
  if (r->positions && ((uintptr_t)r->positions & 3u)) return fail(SDPA_ERR_ALIGN, "positions must be 4-byte aligned");
  if (r->positions && r->axes > 1 && r->pos_stride < 0)
    return fail(SDPA_ERR_STRIDE, "pos_stride %lld < 0", (long long)r->pos_stride);
  int64_t sum = 0;
  for (int a = 0; a < kRopeAxes; ++a) {
    out->sec_end[a] = INT_MAX;
    if (a >= r->axes) continue;
    if (r->sections[a] < 0) return fail(SDPA_ERR_ARG, "sections[%d] = %d < 0", a, r->sections[a]);
    sum += r->sections[a];
    out->sec_end[a] = (int)std::min<int64_t>(sum, INT_MAX);
  }
  if (sum != r->rot_dims / 2)
    return fail(SDPA_ERR_ARG, "sections sum to %lld, not to rot_dims / 2 = %d", (long long)sum, r->rot_dims / 2);
  out->table = (const float2*)r->table;
  out->P = r->table_rows;
  out->half = r->rot_dims / 2;
  out->axes = r->axes;
  out->pos = r->positions;
  out->pos_stride = r->pos_stride;
  out->inverse = inverse ? 1 : 0;
  return SDPA_OK;
}

// What the entries that walk a segment table have in common.
sdpa_status check_step(int64_t T, int Hq, int Hkv, int D, int S, int64_t rows, int cols, int window,
                       const int32_t* seq_info, const int32_t* seg_mode) {
  sdpa_status st = check_common(T, Hq, Hkv, D, S, rows, cols, window, 1.f);
  if (st) return st;
  if (Hq + 2 * (int64_t)Hkv > kMaxHeads) return fail(SDPA_ERR_SHAPE, "more than %d heads", kMaxHeads);
  if (!seq_info && S > 0) return fail(SDPA_ERR_NULL, "seq_info is NULL");
  if (!aligned16(seq_info) || !aligned16(seg_mode))
    return fail(SDPA_ERR_ALIGN, "seq_info and seg_mode must be 16-byte aligned");
  return SDPA_OK;
}

// Warps that share a row of `passes` passes: enough for 24 warps on every SM, at most one a pass.
int row_parts(int64_t T, int passes, int sms) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(passes, 24 * (int64_t)sms / std::max<int64_t>(T, 1)));
}

// A step's kernel: `passes` of a row, or 0 for the read-back, whose CTAs take whole rows.  The grid is
// one wave of three CTAs per SM, or as many CTAs as give each of their warps one pass.
sdpa_status launch_step(const void* f, StepArgs& A, int passes, cudaStream_t stream, const char* what) {
  if (A.T == 0) return SDPA_OK;
  int sms = 0;
  sdpa_status st = device_sms(&sms);
  if (st) return st;
  const int64_t wave = 3 * (int64_t)sms;
  int64_t grid;
  if (passes > 0) {
    const int64_t all = A.T * passes;
    const int64_t per = std::max<int64_t>(kRopeThreads / 32, (all + wave - 1) / wave);
    if (per > INT_MAX) return fail(SDPA_ERR_SHAPE, "%lld rows of %d heads", (long long)A.T, A.Hq + 2 * A.Hkv);
    A.per = (int)per;
    grid = (all + per - 1) / per;
  } else {
    A.cr = (int)std::max<int64_t>(1, std::min<int64_t>(kStepRows, A.T / wave));
    grid = (A.T + A.cr - 1) / A.cr;
  }
  void* args[] = {(void*)&A};
  cudaError_t e = cudaLaunchKernel(f, dim3((unsigned)grid), dim3(kRopeThreads), args, 0, stream);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return SDPA_OK;
}

// The 8-bit append: CTAs for blocks of keys and values, then CTAs for queries (`q_passes` of a row).  A run of
// rows holds the beginnings of about T / 16 + S blocks over the whole table, and a CTA takes the rows of about one
// block; where that leaves SMs idle, CTAs share a run's heads, down to one (head, K or V) a warp.
sdpa_status launch_step_q8(const void* f, StepArgs& A, int q_passes, cudaStream_t stream) {
  if (A.T == 0) return SDPA_OK;
  int sms = 0;
  sdpa_status st = device_sms(&sms);
  if (st) return st;
  const int64_t wave = 3 * (int64_t)sms, warps = kRopeThreads / 32;
  const int64_t blocks = A.T / kPackedRows + std::min<int64_t>(A.S, A.T) + 1;
  A.cr = (int)std::min<int64_t>(kStepRows, (A.T + blocks - 1) / blocks);
  const int64_t runs = (A.T + A.cr - 1) / A.cr;
  A.kv_parts = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>((2 * (int64_t)A.Hkv + warps - 1) / warps, A.Hkv), wave / runs));
  const int64_t kv = A.S > 0 ? runs * A.kv_parts : 0;
  const int64_t all = A.T * q_passes, per = std::max<int64_t>(warps, (all + wave - 1) / wave);
  const int64_t grid = kv + (all + per - 1) / per;
  if (per > INT_MAX || grid > INT_MAX) return fail(SDPA_ERR_SHAPE, "%lld rows of %d heads", (long long)A.T, A.Hq + 2 * A.Hkv);
  A.kv_ctas = (int)kv;
  A.per = (int)per;
  void* args[] = {(void*)&A};
  cudaError_t e = cudaLaunchKernel(f, dim3((unsigned)grid), dim3(kRopeThreads), args, 0, stream);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "rotated 8-bit append launch: %s", cudaGetErrorString(e));
  return SDPA_OK;
}

sdpa_status rope_append(const void* q, int64_t q_rs, int64_t q_hs, const void* k, int64_t k_rs, int64_t k_hs,
                        const void* v, int64_t v_rs, int64_t v_hs, int64_t T, int Hq, int Hkv, int D,
                        const sdpa_rotation* rotation, void* k_store, void* v_store, const PackedStore* packed, int bits,
                        int64_t rows, int cols, const int32_t* seq_info, const int32_t* seg_mode, int S, int window, void* q_out,
                        int64_t o_rs, int64_t o_hs, int32_t* status_dev, void* stream) {
  set_last_error("");
  sdpa_status st = check_step(T, Hq, Hkv, D, S, rows, cols, window, seq_info, seg_mode);
  if (st) return st;
  StepArgs A{};
  if ((st = take_rotation(rotation, T, D, true, 0, &A.r))) return st;
  if (T > 0 && (!q || !k || !v || !q_out)) return fail(SDPA_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out))
    return fail(SDPA_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (bad_strides(q_rs, q_hs) || bad_strides(k_rs, k_hs) || bad_strides(v_rs, v_hs) || bad_strides(o_rs, o_hs))
    return fail(SDPA_ERR_STRIDE, "row/head strides must be non-negative multiples of 8 elements");
  if (packed) {
    if ((st = check_packed_store(*packed, bits, rows))) return st;
    A.q4 = *packed;
  } else {
    if (!k_store || !v_store) return fail(SDPA_ERR_NULL, "a store pointer is NULL");
    if (!aligned16(k_store) || !aligned16(v_store)) return fail(SDPA_ERR_ALIGN, "stores must be 16-byte aligned");
  }
  A.seq_info = seq_info;
  A.seg_mode = seg_mode;
  A.S = S;
  A.window = window;
  A.cols = cols;
  A.Hq = Hq;
  A.Hkv = Hkv;
  A.T = T;
  A.rows = rows;
  A.q = (const __nv_bfloat16*)q;
  A.k = (const __nv_bfloat16*)k;
  A.v = (const __nv_bfloat16*)v;
  A.q_rs = q_rs;
  A.q_hs = q_hs;
  A.k_rs = k_rs;
  A.k_hs = k_hs;
  A.v_rs = v_rs;
  A.v_hs = v_hs;
  A.q_out = (__nv_bfloat16*)q_out;
  A.o_rs = o_rs;
  A.o_hs = o_hs;
  A.k_store = (__nv_bfloat16*)k_store;
  A.v_store = (__nv_bfloat16*)v_store;
  A.status_dev = status_dev;
  const int hpp = rope_heads_per_pass(D), q_passes = (Hq + hpp - 1) / hpp;
  if (bits == 8)
    return launch_step_q8(rope_append_q8_kernel_ptr(D, rotation->interleaved != 0), A, q_passes, (cudaStream_t)stream);
  return launch_step(rope_append_kernel_ptr(D, rotation->interleaved != 0, bits == 4), A,
                     q_passes + 2 * ((Hkv + hpp - 1) / hpp), (cudaStream_t)stream, "rotated append");
}

// Rows of a segment table read back from a store of codes.
sdpa_status unpack(const PackedStore& store, int bits, int64_t rows, int cols, int Hkv, int D, const int32_t* seq_info,
                   const int32_t* seg_mode, int S, int window, int64_t T, void* k_out, void* v_out, int64_t o_rs,
                   int64_t o_hs, int32_t* status_dev, void* stream) {
  sdpa_status st = check_step(T, Hkv, Hkv, D, S, rows, cols, window, seq_info, seg_mode);
  if (st) return st;
  StepArgs A{};
  A.q4 = store;
  if ((st = check_packed_store(store, bits, rows))) return st;
  if (T > 0 && (!k_out || !v_out)) return fail(SDPA_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(SDPA_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (bad_strides(o_rs, o_hs))
    return fail(SDPA_ERR_STRIDE, "row/head strides must be non-negative multiples of 8 elements");
  A.seq_info = seq_info;
  A.seg_mode = seg_mode;
  A.S = S;
  A.window = window;
  A.cols = cols;
  A.Hkv = Hkv;
  A.T = T;
  A.rows = rows;
  A.k_out = (__nv_bfloat16*)k_out;
  A.v_out = (__nv_bfloat16*)v_out;
  A.o_rs = o_rs;
  A.o_hs = o_hs;
  A.status_dev = status_dev;
  return launch_step(bits == 8 ? q8_unpack_kernel_ptr(D) : q4_unpack_kernel_ptr(D), A, 0, (cudaStream_t)stream,
                     bits == 8 ? "8-bit unpack" : "4-bit unpack");
}

}  // namespace
}  // namespace sdpa

using namespace sdpa;

extern "C" {

sdpa_status sdpa_rope(const void* x, int64_t T, int H, int D, int64_t x_row_stride, int64_t x_head_stride,
                      const sdpa_rotation* rotation, int inverse, void* out, int64_t o_row_stride,
                      int64_t o_head_stride, int32_t* status_dev, void* stream) {
  set_last_error("");
  if (T < 0 || T > INT_MAX || H <= 0 || H > kMaxHeads) return fail(SDPA_ERR_SHAPE, "bad sizes: T=%lld H=%d", (long long)T, H);
  if (D != 64 && D != 128 && D != 256) return fail(SDPA_ERR_HEAD_DIM, "head dim %d not in {64,128,256}", D);
  RopeRowsArgs A{};
  sdpa_status st = take_rotation(rotation, T, D, false, inverse, &A.r);
  if (st) return st;
  if (T > 0 && (!x || !out)) return fail(SDPA_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(x) || !aligned16(out)) return fail(SDPA_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (bad_strides(x_row_stride, x_head_stride) || bad_strides(o_row_stride, o_head_stride))
    return fail(SDPA_ERR_STRIDE, "row/head strides must be non-negative multiples of 8 elements");
  if (T == 0) return SDPA_OK;
  int sms = 0;
  if ((st = device_sms(&sms))) return st;
  A.x = (const __nv_bfloat16*)x;
  A.out = (__nv_bfloat16*)out;
  A.x_rs = x_row_stride;
  A.x_hs = x_head_stride;
  A.o_rs = o_row_stride;
  A.o_hs = o_head_stride;
  A.T = T;
  A.H = H;
  A.status_dev = status_dev;
  const int hpp = rope_heads_per_pass(D);
  A.parts = row_parts(T, (H + hpp - 1) / hpp, sms);
  const int64_t warps = T * A.parts;
  const int64_t blocks = std::min<int64_t>((warps * 32 + kRopeThreads - 1) / kRopeThreads, (int64_t)sms * 3);
  void* args[] = {(void*)&A};
  cudaError_t e = cudaLaunchKernel(rope_kernel_ptr(D, rotation->interleaved != 0), dim3((unsigned)blocks),
                                   dim3(kRopeThreads), args, 0, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "rotation launch: %s", cudaGetErrorString(e));
  return SDPA_OK;
}

sdpa_status sdpa_rope_append(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k_new,
                             int64_t k_row_stride, int64_t k_head_stride, const void* v_new, int64_t v_row_stride,
                             int64_t v_head_stride, int64_t T, int Hq, int Hkv, int D,
                             const sdpa_rotation* rotation, void* k_store, void* v_store, int64_t rows, int cols,
                             const int32_t* seq_info, const int32_t* seg_mode, int S, int window, void* q_out,
                             int64_t o_row_stride, int64_t o_head_stride, int32_t* status_dev, void* stream) {
  return rope_append(q, q_row_stride, q_head_stride, k_new, k_row_stride, k_head_stride, v_new, v_row_stride,
                     v_head_stride, T, Hq, Hkv, D, rotation, k_store, v_store, nullptr, 16, rows, cols, seq_info,
                     seg_mode, S, window, q_out, o_row_stride, o_head_stride, status_dev, stream);
}

sdpa_status sdpa_rope_append_fourbit(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k_new,
                                int64_t k_row_stride, int64_t k_head_stride, const void* v_new,
                                int64_t v_row_stride, int64_t v_head_stride, int64_t T, int Hq, int Hkv, int D,
                                const sdpa_rotation* rotation, const sdpa_q4_store* store, int64_t rows, int cols,
                                const int32_t* seq_info, const int32_t* seg_mode, int S, int window, void* q_out,
                                int64_t o_row_stride, int64_t o_head_stride, int32_t* status_dev, void* stream) {
  set_last_error("");
  if (!store) return fail(SDPA_ERR_NULL, "store is NULL");
  const PackedStore q4{store->k_codes, store->k_scales, store->v_codes, store->v_scales};
  return rope_append(q, q_row_stride, q_head_stride, k_new, k_row_stride, k_head_stride, v_new, v_row_stride,
                     v_head_stride, T, Hq, Hkv, D, rotation, nullptr, nullptr, &q4, 4, rows, cols, seq_info, seg_mode, S,
                     window, q_out, o_row_stride, o_head_stride, status_dev, stream);
}

sdpa_status sdpa_rope_append_eightbit(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k_new,
                                 int64_t k_row_stride, int64_t k_head_stride, const void* v_new,
                                 int64_t v_row_stride, int64_t v_head_stride, int64_t T, int Hq, int Hkv, int D,
                                 const sdpa_rotation* rotation, const sdpa_q8_store* store, int64_t rows, int cols,
                                 const int32_t* seq_info, const int32_t* seg_mode, int S, int window, void* q_out,
                                 int64_t o_row_stride, int64_t o_head_stride, int32_t* status_dev, void* stream) {
  set_last_error("");
  if (!store) return fail(SDPA_ERR_NULL, "store is NULL");
  const PackedStore q8{store->k_codes, store->k_scales, store->v_codes, store->v_scales};
  return rope_append(q, q_row_stride, q_head_stride, k_new, k_row_stride, k_head_stride, v_new, v_row_stride,
                     v_head_stride, T, Hq, Hkv, D, rotation, nullptr, nullptr, &q8, 8, rows, cols, seq_info, seg_mode, S,
                     window, q_out, o_row_stride, o_head_stride, status_dev, stream);
}

sdpa_status sdpa_fourbit_unpack(const sdpa_q4_store* store, int64_t rows, int cols, int Hkv, int D,
                           const int32_t* seq_info, const int32_t* seg_mode, int S, int window, int64_t T,
                           void* k_out, void* v_out, int64_t o_row_stride, int64_t o_head_stride,
                           int32_t* status_dev, void* stream) {
  set_last_error("");
  if (!store) return fail(SDPA_ERR_NULL, "store is NULL");
  return unpack(PackedStore{store->k_codes, store->k_scales, store->v_codes, store->v_scales}, 4, rows, cols, Hkv, D,
                seq_info, seg_mode, S, window, T, k_out, v_out, o_row_stride, o_head_stride, status_dev, stream);
}

sdpa_status sdpa_eightbit_unpack(const sdpa_q8_store* store, int64_t rows, int cols, int Hkv, int D,
                            const int32_t* seq_info, const int32_t* seg_mode, int S, int window, int64_t T,
                            void* k_out, void* v_out, int64_t o_row_stride, int64_t o_head_stride,
                            int32_t* status_dev, void* stream) {
  set_last_error("");
  if (!store) return fail(SDPA_ERR_NULL, "store is NULL");
  return unpack(PackedStore{store->k_codes, store->k_scales, store->v_codes, store->v_scales}, 8, rows, cols, Hkv, D,
                seq_info, seg_mode, S, window, T, k_out, v_out, o_row_stride, o_head_stride, status_dev, stream);
}

}  // extern "C"
