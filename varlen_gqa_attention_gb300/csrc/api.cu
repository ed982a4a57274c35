// api.cu - the C interface: argument checks, workspace layout, launches.
//
// Every check runs before any CUDA call, so a bad argument never touches the device.  The
// launches are asynchronous and allocation-free, so a call can be captured in a CUDA graph;
// the device scheduler reads the segment table when the graph replays.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "q4.cuh"
#include "q8.cuh"

namespace sdpa {

static thread_local char g_err[512] = "";
static thread_local cudaEvent_t g_ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
static thread_local bool g_ev_on = false;

// Records timing event i on `st`.  Under stream capture the record must become an event
// node of the graph (cudaEventRecordExternal) so that it fires on every replay.
static cudaError_t mark(int i, cudaStream_t st) {
  if (!g_ev_on) return cudaSuccess;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(st, &cs);
  if (e != cudaSuccess) return e;
  return cs == cudaStreamCaptureStatusActive ? cudaEventRecordWithFlags(g_ev[i], st, cudaEventRecordExternal)
                                             : cudaEventRecord(g_ev[i], st);
}
static std::atomic<int> g_policy{SDPA_ROUTE_AUTO};

sdpa_status fail(sdpa_status code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

void set_last_error(const char* msg) { snprintf(g_err, sizeof(g_err), "%s", msg); }

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Per-device launch facts, measured once.
struct DevInfo {
  bool ready = false;
  int sms = 0;
  int splitk_per_sm[3] = {0, 0, 0};  // D = 64, 128, 256
  int packed_per_sm[2][3] = {};  // 4 and 8 bits
  bool prefill_ok[3] = {false, false, false};
};
static std::mutex g_mu;
static DevInfo g_dev[64];

// The kernels of a store of codes.
static const void* packed_splitk_ptr(int bits, int D) { return bits == 8 ? q8_splitk_kernel_ptr(D) : q4_splitk_kernel_ptr(D); }
static const void* packed_direct_ptr(int bits, int D) { return bits == 8 ? q8_direct_kernel_ptr(D) : q4_direct_kernel_ptr(D); }
static const void* packed_tile_ptr(int bits, int D) { return bits == 8 ? q8_tile_kernel_ptr(D) : q4_tile_kernel_ptr(D); }
static int packed_tile_smem(int bits, int D) { return bits == 8 ? q8_tile_smem_bytes(D) : q4_tile_smem_bytes(D); }
static int packed_smem_bytes(int bits, int D) { return bits == 8 ? q8_splitk_smem_bytes(D) : q4_splitk_smem_bytes(D); }

static int d_index(int D) { return D == 64 ? 0 : D == 128 ? 1 : 2; }

static sdpa_status device_info(DevInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(SDPA_ERR_CUDA, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& di = g_dev[dev];
  if (!di.ready) {
    e = cudaDeviceGetAttribute(&di.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "SM count: %s", cudaGetErrorString(e));
    for (int packed = 0; packed < 2; ++packed) {
      e = cudaFuncSetAttribute(sched_kernel_ptr(packed), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)sched_smem_bytes());
      if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "scheduler smem attribute: %s", cudaGetErrorString(e));
    }
    // every kernel of a call asks for the whole shared-memory carveout, so that the SMs keep
    // one L1 / shared split from kernel to kernel (the clone kernel runs alone and keeps the
    // default split, its L1 to itself)
    const void* others[5] = {sched_kernel_ptr(false), sched_small_kernel_ptr(false), append_kernel_ptr(),
                             sched_kernel_ptr(true), sched_small_kernel_ptr(true)};
    for (const void* f : others) {
      e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "carveout attribute: %s", cudaGetErrorString(e));
    }
    const int Ds[3] = {64, 128, 256};
    for (int k = 0; k < 3; ++k) {
      const void* f = splitk_kernel_ptr(Ds[k]);
      const int smem = splitk_smem_bytes(Ds[k]);
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "smem attribute: %s", cudaGetErrorString(e));
      // two split-K CTAs per SM need the whole shared-memory carveout
      e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "carveout attribute: %s", cudaGetErrorString(e));
      int nb = 0;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, f, kSplitkThreads, smem);
      if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "occupancy: %s", cudaGetErrorString(e));
      di.splitk_per_sm[k] = nb > 0 ? nb : 1;
      for (int bits = 4; bits <= 8; bits += 4) {
        if (Ds[k] <= 128) {
          const void* tile = packed_tile_ptr(bits, Ds[k]);
          e = cudaFuncSetAttribute(tile, cudaFuncAttributeMaxDynamicSharedMemorySize, packed_tile_smem(bits, Ds[k]));
          if (e == cudaSuccess) e = cudaFuncSetAttribute(tile, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
          if (e != cudaSuccess)
            return fail(SDPA_ERR_CUDA, "%d-bit tile kernel attributes: %s", bits, cudaGetErrorString(e));
        }
        const void* few = packed_splitk_ptr(bits, Ds[k]);
        const int few_smem = packed_smem_bytes(bits, Ds[k]);
        for (const void* f : {few, packed_direct_ptr(bits, Ds[k])}) {
          e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem);
          if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
          if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "%d-bit kernel attributes: %s", bits, cudaGetErrorString(e));
        }
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&nb, few, kPackedThreads, few_smem);
        if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "occupancy: %s", cudaGetErrorString(e));
        di.packed_per_sm[bits / 8][k] = nb > 0 ? nb : 1;
      }
      e = cudaFuncSetAttribute(combine_pair_kernel_ptr(Ds[k]), cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "carveout attribute: %s", cudaGetErrorString(e));
      for (int q = 0; q < 2; ++q) {
        e = cudaFuncSetAttribute(combine_kernel_ptr(Ds[k], q), cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "carveout attribute: %s", cudaGetErrorString(e));
      }
      for (int f16 = 0; f16 < 2 && e == cudaSuccess; ++f16) {
        const void* pf = prefill_kernel_ptr(Ds[k], f16);
        e = cudaFuncSetAttribute(pf, cudaFuncAttributeMaxDynamicSharedMemorySize, prefill_smem_bytes(Ds[k]));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(pf, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
      }
      di.prefill_ok[k] = e == cudaSuccess;
      if (e != cudaSuccess) cudaGetLastError();  // leave no sticky error; split-K covers it
    }
    di.ready = true;
  }
  *out = di;
  return SDPA_OK;
}

// cuTensorMapEncodeTiled, fetched from the driver once (no link against libcuda).
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)p;
    else
      cudaGetLastError();
  });
  return fn;
}

// TMA descriptors of q [T, Hq, D] (box: 64 dims x group heads x 128/group rows, i.e. one
// 128-row tile of packed (row, head) pairs) and of the stores [rows, cols, Hkv, D] (box:
// 64 dims x 1 head x 1 column x `bn` rows), all with 128-byte swizzle.
static bool make_tensor_maps(const void* q, int64_t T, int Hq, int D, int64_t q_rs, int64_t q_hs,
                             const void* k, const void* v, int64_t rows, int cols, int Hkv, int group,
                             int bn, bool v_f16, CUtensorMap* mq, CUtensorMap* mk, CUtensorMap* mv) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc || T <= 0 || q_hs <= 0 || q_rs <= 0) return false;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint64_t qdim[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T};
  const cuuint64_t qstr[2] = {(cuuint64_t)q_hs * 2, (cuuint64_t)q_rs * 2};
  const cuuint32_t qbox[3] = {64, (cuuint32_t)group, (cuuint32_t)(kPrefillRows / group)};
  if (enc(mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)q, qdim, qstr, qbox, es,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  const cuuint64_t kdim[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t kstr[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2, (cuuint64_t)cols * Hkv * D * 2};
  const cuuint32_t kbox[4] = {64, 1, 1, (cuuint32_t)bn};
  for (int w = 0; w < 2; ++w) {
    if (enc(w ? mv : mk, w && v_f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void*)(w ? v : k), kdim, kstr, kbox, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

// TMA descriptors of an 8-bit store's codes [cols * Hkv, rows, D]: boxes of 16 rows and of q8_box_rows, 128 bytes wide
// (64 at D = 64), swizzled over their width.
static bool make_q8_maps(const PackedStore& st, int64_t rows, int cols, int Hkv, int D, Q8AttnArgs* out) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint32_t es[3] = {1, 1, 1};
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)cols * Hkv};
  const cuuint64_t stride[2] = {(cuuint64_t)D, (cuuint64_t)rows * D};
  CUtensorMap* const maps[4] = {&out->k, &out->v, &out->k_box, &out->v_box};
  for (int i = 0; i < 4; ++i) {
    const cuuint32_t box[3] = {(cuuint32_t)std::min(D, 128), (cuuint32_t)(i < 2 ? kPackedRows : q8_box_rows(D)), 1};
    if (enc(maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, i & 1 ? st.vc : st.kc, dim, stride, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

struct Grids {
  int64_t splitk, prefill;
};
static Grids grids_for(const DevInfo& di, int D) {
  Grids g;
  g.splitk = (int64_t)di.sms * di.splitk_per_sm[d_index(D)];
  g.prefill = di.sms;
  return g;
}

// The kernels over codes for the split-K route: the tensor-memory one (packed_tile.cuh), which converts a key once
// for up to 128 packed rows, and the other one (packed_attn.cuh), which converts a key again for every 8. Over the
// 4-bit store, 64 segments over 6144 keys on average, 8 KV heads, D = 128, tensor-memory / other: 16 rows 150 / 131
// us, 24 rows 150 / 303 us; 16 segments of 64 rows over 3100 keys 43 / 100 us.  The host knows how many rows the
// average segment has (empty ones counted): with at most 16 (8 bits, D = 64: 32) it launches the other one, with more
// (of several segments, which may be one chunk and many single tokens) both, and the schedule is the cheaper one's;
// the other leaves at once.  At D = 256 the output of 128 rows leaves no room for the first.
enum class PackedSplit { kFew, kTile, kEither };
static PackedSplit packed_split(int bits, int64_t T, int Hq, int Hkv, int D, int S) {
  const int few = bits == 8 && D == 64 ? 32 : 16;
  if (D > 128 || T * (Hq / Hkv) <= few * (int64_t)std::max(S, 1)) return PackedSplit::kFew;
  return S <= 1 ? PackedSplit::kTile : PackedSplit::kEither;
}
// The tensor-memory kernel's cost of a key for a unit, in those of the other one for 8 rows (full loads: 0.066
// and 0.027 ns at D = 128, 0.054 and 0.015 at D = 64).  Over the 8-bit store, against the other one's 8 rows (the calls
// of tile_cost, common.cuh): 160 us for 24 rows and 177 for 64 at D = 128, 157 for 32 and 165 for 64 at D = 64.
static float packed_tile_ratio(int bits, int D) { return bits == 8 ? (D == 64 ? 3.6f : 2.1f) : D == 64 ? 3.5f : 2.5f; }
static int64_t packed_resident(const DevInfo& di, int bits, int D) {
  return (int64_t)di.sms * di.packed_per_sm[bits / 8][d_index(D)];
}
static SkShape packed_few_shape(const DevInfo& di, int bits, int D) {
  return {kSplitkRows, kSplitkTile, bits == 8 ? kSkQ8Few : kSkQ4Few, packed_resident(di, bits, D)};
}
static SkShape packed_tile_shape(const DevInfo& di) { return {kPackedTileRows, kPackedTileKeys, kSkQ4Tile, di.sms}; }

sdpa_status check_common(int64_t T, int Hq, int Hkv, int D, int S, int64_t rows, int cols, int window,
                         float scale) {
  if (T < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || rows <= 0 || cols <= 0)
    return fail(SDPA_ERR_SHAPE, "bad sizes: T=%lld S=%d Hq=%d Hkv=%d rows=%lld cols=%d",
                (long long)T, S, Hq, Hkv, (long long)rows, cols);
  if (T > INT32_MAX || rows > INT32_MAX || (int64_t)Hq * T > ((int64_t)1 << 40))
    return fail(SDPA_ERR_SHAPE, "T or rows beyond 2^31-1");
  if (D != 64 && D != 128 && D != 256) return fail(SDPA_ERR_HEAD_DIM, "head dim %d not in {64,128,256}", D);
  if (Hq % Hkv != 0 || Hq / Hkv > 128)
    return fail(SDPA_ERR_GQA, "Hq=%d is not a multiple of Hkv=%d (group <= 128)", Hq, Hkv);
  if (window < 0) return fail(SDPA_ERR_ARG, "window %d < 0", window);
  if (!std::isfinite(scale)) return fail(SDPA_ERR_ARG, "scale is not finite");
  return SDPA_OK;
}

sdpa_status check_tensors(const void* q, const void* k, const void* v, void* out, const int32_t* seq_info,
                          int S, int64_t q_rs, int64_t q_hs, int64_t o_rs, int64_t o_hs) {
  if (!q || !k || !v || !out || (!seq_info && S > 0)) return fail(SDPA_ERR_NULL, "a required pointer is NULL");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || (seq_info && !aligned16(seq_info)))
    return fail(SDPA_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (q_rs % 8 || q_hs % 8 || o_rs % 8 || o_hs % 8 || q_rs < 0 || q_hs < 0 || o_rs < 0 || o_hs < 0)
    return fail(SDPA_ERR_STRIDE, "row/head strides must be non-negative multiples of 8 elements");
  return SDPA_OK;
}

sdpa_status check_packed_store(const PackedStore& st, int bits, int64_t rows) {
  if (!st.kc || !st.ks || !st.vc || !st.vs) return fail(SDPA_ERR_NULL, "a %d-bit store pointer is NULL", bits);
  if (!aligned16(st.kc) || !aligned16(st.vc) || (bits == 4 && (!aligned16(st.ks) || !aligned16(st.vs))))
    return fail(SDPA_ERR_ALIGN, "%d-bit store pointers must be 16-byte aligned", bits);
  if (rows % kPackedRows)
    return fail(SDPA_ERR_SHAPE, "a %d-bit store has a multiple of %d rows, not %lld", bits, kPackedRows,
                (long long)rows);
  return SDPA_OK;
}

struct TensorMaps {
  CUtensorMap q, k, v;
};

// A call over a store of codes: the kernels' arguments, of whichever store it is.
struct PackedCall {
  int bits;
  PackedStore st;
  Q8AttnArgs q8;
  Q4AttnArgs q4;
  void* args() { return bits == 8 ? (void*)&q8 : (void*)&q4; }
};

// Launch with programmatic stream serialisation (the kernel waits in-kernel for its
// predecessor), except while the timing hook records events between the kernels: an event
// between two kernels would only serialise them again, and each kernel is then timed alone.
static cudaError_t launch_k(const void* f, unsigned grid, unsigned block, void** args, size_t smem,
                            cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  if (pdl && !g_ev_on) {
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelExC(&cfg, f, args);
}

// CTAs that share a (token, KV head) pair's keys when a call over codes takes the kernel without a schedule; 0 when
// it does not.  It does where a CTA's share of the longest range possible is short, and the table has an entry for
// every token or more, or the pairs' CTAs all fit the SMs at once.  The host sees neither lengths nor empty entries:
// the longest range is the store's rows (or a call-wide window; 128 keys, 4/1 heads, D = 64: 6.2 us in a store of 128
// rows, 8.3 in one of 32768, where a cluster of 8 is taken, 14.4 scheduled), and an empty entry counts as a token of
// its own.  256 entries, one of them 200 tokens over 2048 keys, 20 single tokens and the others empty: 117 us, 66
// without the empty ones (256 single tokens of 2048 keys 140 / 209, which is why the rule is so).  The shares are
// halved while there are SMs for them and more than kDirectPart keys in each.  In us, direct / scheduled, 4 bits,
// 32/8 heads, D = 128, all ranges full: 1 token 512 keys 7.0 / 14.4, 16384 keys 15.8 / 19.4; 8 tokens 64 keys 6.0 /
// 13.0, 2048 keys 10.3 / 18.8, 16384 keys 40 / 45; 32 tokens 512 keys 8.9 / 22.6, 4096 keys 38 / 49; 64 tokens 2048
// keys 41 / 62; two segments of 16 tokens 1024 keys 13 / 26, 4096 keys 36 / 28. Where lengths differ the call waits
// for its longest: lengths evenly spread up to the limit (32 tokens of 4096 keys, 34.5 / 33.6; with 16/2 heads of
// 8192, 21 / 24, of 16384 beyond it 36 / 30; 16 tokens at D = 256 of 4096 30 / 32, of 8192 52 / 47). Over the 8-bit
// store, all ranges full and evenly spread ones: 32/8 heads, D = 128: 32 tokens of 4096 keys 46 / 58 and 39 / 41, of
// 8192 beyond it 83 / 94 and 66 / 61, 16 of 16384 83 / 92 and 65 / 53; with 16/2 heads 32 of 8192 29 / 39 and 22 /
// 25, of 16384 47 / 56 and 41 / 42.  D = 64, 32/8 heads: 32 of 8192 48 / 57 and 36 / 37, 16 of 16384 beyond it 49 /
// 57 and 35 / 31. D = 256, 16/4 heads: 16 of 4096 32 / 39 and 25 / 27, of 8192 51 / 57 and 42 / 39, 32 of 4096 50 /
// 59 and 40 / 38; clusters of 8, whose CTAs are then few: 4 of 8192 26 / 26 and 17 / 22, of 16384 beyond it 45 / 39
// and 43 / 32.  Segments of several tokens: 2 of 16 tokens 1024 keys 15 / 28, beyond it 4096 keys 38 / 30.
// Shares halved until the CTAs make two waves: 8 bits, 32 tokens of 8192 keys, 16/2 heads, full 27.4 us in one wave, 36.6 in
// two, evenly spread 20.8 / 26.0 (one of 8192 keys among ones of 64, 17.9 / 14.6).
constexpr int64_t kDirectPart = 128;
static int packed_direct_parts(const DevInfo& di, int bits, int64_t T, int Hq, int Hkv, int D, int S, int64_t rows,
                               int causal, int window, const int32_t* seg_mode) {
  if (g_policy.load() != SDPA_ROUTE_AUTO || Hq / Hkv > kSplitkRows || S > kPackedDirectSegs) return 0;
  const int64_t pairs = T * Hkv, resident = packed_resident(di, bits, D);
  if (T > S && pairs > resident) return 0;
  int64_t keys = rows;  // that a row may see
  if (window > 0 && !seg_mode) keys = std::min<int64_t>(keys, causal ? window : T + window - 1);
  int parts = 1;
  while (parts < 8 && 2 * parts * pairs <= resident && keys > kDirectPart * parts) parts *= 2;
  int64_t share = T <= S && (D == 64 || (D == 128 && parts <= 2)) ? 4096 : 2048;
  if (bits == 8 && T <= S) {
    if (D == 64) share = parts == 1 ? 8192 : 4096;
    if (D == 128) share = parts == 8 ? 2048 : 4096;
    if (D == 256) share = parts == 8 ? 1024 : 2048;
  }
  return keys <= share * parts ? parts : 0;
}

// The prefill route over codes: a store's columns are staged first, which many rows have to pay for, and the route it
// competes with is the tensor-memory kernel of packed_tile.cuh, where that one runs.  Split-K / prefill, 4 bits, 32/8
// heads, D = 128, in us: one segment over 4096 keys, 128 rows a head 37 / 39, 256 rows 48 / 47, 512 rows 70 / 65,
// 2048 rows 168 / 136; 128 rows over 32768 keys 92 / 143, 512 rows 292 / 265; four segments of 128 rows over 4096
// keys 73 / 102, sixteen 206 / 259.  At D = 256 the split-K kernel converts a key again for every 8 rows: 64 rows a
// head over 4096 keys 76 / 45. So the bf16 entry's thresholds hold where the tensor-memory one is not launched, and
// 512 rows where the schedule takes the other one: 64 tokens over 16384 to 32768 keys beside 250 over 32768 842 / 579
// us (fewer rows do not pay for the launches when there are none, 5 us).
constexpr int kTilePrefillRows = 1024;
static int packed_prefill_min_rows(PackedSplit sp) {
  return sp == PackedSplit::kFew ? kPrefillRows : sp == PackedSplit::kEither ? 512 : kTilePrefillRows;
}
static float packed_prefill_min_work(PackedSplit sp) { return sp == PackedSplit::kFew ? kPrefillMinWork : 4 * kPrefillMinWork; }
// Packed rows of a call's longest segment when none is empty.
static int64_t packed_longest(int64_t T, int group, int S) { return std::max<int64_t>(1, T - std::max(S, 1) + 1) * group; }
// Columns a call over codes stages in 16 bits for the prefill kernel: one per segment that can have
// packed_prefill_min_rows, as far as 2 GiB of workspace hold them (at least one while that takes at most 8 GiB); none
// when the automatic route cannot reach packed_prefill_min_work.  Depends on sizes and the route policy only.
static int64_t stage_bytes_per_column(int64_t rows, int Hkv, int D) { return rows * Hkv * D * 2; }
static int packed_stage_cols(int bits, int64_t T, int Hq, int Hkv, int D, int S, int64_t rows) {
  const int policy = g_policy.load();
  const int group = Hq / Hkv;
  if (policy == SDPA_ROUTE_SPLITK || group > kPrefillRows || kPrefillRows % group || S <= 0 || T <= 0) return 0;
  const int64_t packed = T * group;
  int64_t n = S;
  if (policy == SDPA_ROUTE_AUTO) {
    const PackedSplit sp = packed_split(bits, T, Hq, Hkv, D, S);
    if (packed_longest(T, group, S) < packed_prefill_min_rows(sp) ||
        (double)packed * Hkv * D * (double)rows < (double)packed_prefill_min_work(sp))
      return 0;
    n = std::min<int64_t>(n, packed / packed_prefill_min_rows(sp));
  }
  const int64_t col = 2 * stage_bytes_per_column(rows, Hkv, D);  // K and V
  if (col > (8ll << 30)) return 0;
  return (int)std::min<int64_t>(n, std::max<int64_t>(1, (2ll << 30) / col));
}

// Whether a call may route segments to the prefill kernel: not under the split-K policy, and
// (automatic routing) not when no segment can have pf_min_rows packed rows or the
// call cannot hold pf_min_work of prefill work: that is at most packed rows * Hkv * D *
// the longest needed key span, which is at most the store's rows (longer spans are invalid)
// and, with a call-wide window, T + window - 1.  The scheduler takes the result as
// prefill_ok, so it never routes work to a prefill kernel that is not launched.
static bool prefill_launch(const SchedArgs& sa, int64_t T) {
  if (sa.policy == SDPA_ROUTE_SPLITK) return false;
  if (sa.policy == SDPA_ROUTE_PREFILL) return true;
  const int64_t packed = T * sa.group;
  int64_t span_max = sa.rows;
  if (!sa.seg_mode && sa.window > 0) span_max = std::min<int64_t>(span_max, T + sa.window - 1);
  return packed >= sa.pf_min_rows && (double)packed * sa.Hkv * sa.D * (double)span_max >= (double)sa.pf_min_work;
}

static sdpa_status launch_all(const SchedArgs& sa, const AttnArgs& aa, int D, const Grids& g,
                              const TensorMaps& tm, const AppendArgs* ap, PackedCall* packed,
                              const PackedStageArgs* stage, cudaStream_t st) {
  cudaError_t e = mark(0, st);
  if (e == cudaSuccess) {
    e = launch_sched(sa, st);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "scheduler launch: %s", cudaGetErrorString(e));
  }
  if (e == cudaSuccess && ap && sa.S > 0) {
    // the step's new keys and values, between the scheduler (whose segment records say
    // which segments are live) and the attention kernels that read them
    void* args[] = {(void*)ap};
    const int64_t per_seg = (aa.T + sa.S - 1) / sa.S;
    const int64_t chunks = per_seg * ap->Hkv * (ap->D / 8);
    const unsigned gy = (unsigned)std::min<int64_t>(256, std::max<int64_t>(1, chunks / (4 * kAppendThreads)));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)sa.S, gy);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    if (!g_ev_on) {
      cfg.attrs = at;
      cfg.numAttrs = 1;
    }
    e = cudaLaunchKernelExC(&cfg, append_kernel_ptr(), args);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
  }
  if (e == cudaSuccess) e = mark(1, st);
  // The prefill kernel is launched when the call's schedule may use it (prefill_ok, see
  // prefill_launch).  Chained to the scheduler (programmatic dependent launch: its launch
  // overlaps the scheduler) when the average segment fills less than one tile, so that the
  // launch is most likely empty; launched after the scheduler otherwise (measured: the
  // chained launch saves ~6 us on a decode step whose prefill kernel has nothing to do, and
  // costs ~5 us on prefill steps of a few tiles per CTA).
  const int64_t rows_packed = aa.T * aa.group;
  const bool pf_possible = sa.prefill_ok;
  if (e == cudaSuccess && pf_possible && stage) {
    void* args[] = {(void*)stage};
    const int64_t chunks = sa.rows_pf * stage->Hkv * (D / 8);  // of one column
    const int64_t most = std::max<int64_t>(1, 8 * g.prefill / stage->pf_cols);
    const int64_t per = std::max<int64_t>(1, std::min<int64_t>(most, chunks / (4 * kPackedStageThreads)));
    e = launch_k(packed->bits == 8 ? q8_stage_kernel_ptr(D) : q4_stage_kernel_ptr(D), (unsigned)(per * stage->pf_cols),
                 kPackedStageThreads, args, 0, st, true);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "column staging launch: %s", cudaGetErrorString(e));
  }
  if (e == cudaSuccess && pf_possible) {
    AttnArgs pa = aa;
    pa.rows = sa.rows_pf;
    void* args[] = {(void*)&pa, (void*)&tm.q, (void*)&tm.k, (void*)&tm.v};
    const bool chained = rows_packed < (int64_t)kPrefillRows * std::max(sa.S, 1);
    e = launch_k(prefill_kernel_ptr(D, packed != nullptr), (unsigned)g.prefill, prefill_block_threads(D), args,
                 prefill_smem_bytes(D), st, chained);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "prefill launch: %s", cudaGetErrorString(e));
  }
  if (e == cudaSuccess) e = mark(2, st);
  if (e == cudaSuccess && packed) {
    void* args[] = {packed->args()};
    const int smem = packed_smem_bytes(packed->bits, D);
    if (sa.sk_choice || sa.sk[0].rows == kSplitkRows)
      e = launch_k(packed_splitk_ptr(packed->bits, D), (unsigned)sa.sk[0].grid, kPackedThreads, args, smem, st, true);
    if (e == cudaSuccess && (sa.sk_choice || sa.sk[0].rows == kPackedTileRows))
      e = launch_k(packed_tile_ptr(packed->bits, D), (unsigned)sa.sk[1].grid, kPackedTileThreads, args,
                   packed_tile_smem(packed->bits, D), st, true);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "%d-bit split-K launch: %s", packed->bits, cudaGetErrorString(e));
  } else if (e == cudaSuccess) {
    void* args[] = {(void*)&aa};
    e = launch_k(splitk_kernel_ptr(D), (unsigned)g.splitk, kSplitkThreads, args, splitk_smem_bytes(D), st, true);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "split-K launch: %s", cudaGetErrorString(e));
  }
  if (e == cudaSuccess) e = mark(3, st);
  if (e == cudaSuccess && aa.T > 0) {
    void* args[] = {(void*)&aa};
    const int64_t warps = aa.T * aa.Hq;
    const int64_t blocks = std::min<int64_t>((warps * 32 + 255) / 256, 8 * (int64_t)g.prefill);
    // calls over codes with few pairs: a CTA each, as many as the SMs hold at once
    if (packed && warps <= 8 * (int64_t)g.prefill)
      e = launch_k(combine_pair_kernel_ptr(D), (unsigned)warps, 256, args, 0, st, true);
    else
      e = launch_k(combine_kernel_ptr(D, packed != nullptr), (unsigned)blocks, 256, args, 0, st, true);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "combine launch: %s", cudaGetErrorString(e));
  }
  if (e == cudaSuccess) e = mark(4, st);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "timing event: %s", cudaGetErrorString(e));
  return SDPA_OK;
}

static sdpa_status run(const void* q, int64_t T, int Hq, int D, int64_t q_rs, int64_t q_hs,
                       const void* k, const void* v, int64_t rows, int cols, int Hkv,
                       const int32_t* seq_info, int S, const int32_t* inl, int causal, int window,
                       float scale, void* out, int64_t o_rs, int64_t o_hs, void* ws, size_t ws_bytes,
                       int32_t* status_dev, void* stream, const AppendArgs* ap = nullptr,
                       const int32_t* seg_mode = nullptr, PackedCall* packed = nullptr) {
  g_err[0] = 0;
  sdpa_status st = check_common(T, Hq, Hkv, D, S, rows, cols, window, scale);
  if (st) return st;
  const int bits = packed ? packed->bits : 16;
  if (packed && (st = check_packed_store(packed->st, bits, rows))) return st;
  if (bits == 8 && (int64_t)cols * Hkv > INT32_MAX)
    return fail(SDPA_ERR_SHAPE, "an 8-bit store of %d columns of %d heads", cols, Hkv);
  if (packed && T == 0) return SDPA_OK;
  // the dense entry passes its one segment by value: no table pointer to check
  if ((st = check_tensors(q, k, v, out, seq_info, inl ? 0 : S, q_rs, q_hs, o_rs, o_hs))) return st;
  if (!ws) return fail(SDPA_ERR_WORKSPACE, "workspace is NULL");
  if ((uintptr_t)ws % 256) return fail(SDPA_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (seg_mode && !aligned16(seg_mode)) return fail(SDPA_ERR_ALIGN, "seg_mode must be 16-byte aligned");

  DevInfo di;
  if ((st = device_info(&di))) return st;
  Grids g = grids_for(di, D);
  PackedSplit sp = PackedSplit::kFew;
  SkShape few{kSplitkRows, kSplitkTile, kSkBf16, g.splitk}, tile = packed_tile_shape(di);
  if (packed) {
    sp = packed_split(bits, T, Hq, Hkv, D, S);
    few = packed_few_shape(di, bits, D);
    g.splitk = few.grid;
  }
  Workspace W;
  size_t need = layout_workspace((char*)ws, T, Hq, Hkv, D, S, g.splitk, g.prefill, &W, true,
                                 packed && D <= 128 ? &tile : nullptr);
  if (ws_bytes < need)
    return fail(SDPA_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  const int parts =
      packed ? packed_direct_parts(di, bits, T, Hq, Hkv, D, S, rows, causal, window, S > 0 ? seg_mode : nullptr) : 0;
  PackedStageArgs sg{};
  if (packed && parts == 0) {  // as many staged columns as the workspace holds
    const int64_t col = stage_bytes_per_column(rows, Hkv, D);  // (a multiple of 256)
    sg.pf_cols = (int)std::min<int64_t>(packed_stage_cols(bits, T, Hq, Hkv, D, S, rows), (int64_t)(ws_bytes - need) / (2 * col));
    sg.k = (__nv_bfloat16*)((char*)ws + need);
    sg.v = (__half*)((char*)ws + need + col * sg.pf_cols);
  }

  SchedArgs sa{};
  sa.seq_info = seq_info;
  sa.seg_mode = S > 0 ? seg_mode : nullptr;
  sa.S = S;
  sa.use_inline = inl != nullptr;
  if (inl)
    for (int i = 0; i < 4; ++i) sa.inl[i] = inl[i];
  sa.T = T;
  sa.rows = rows;
  sa.cols = cols;
  sa.Hkv = Hkv;
  sa.group = Hq / Hkv;
  sa.causal = causal ? 1 : 0;
  sa.window = window;
  sa.D = D;
  sa.policy = g_policy.load();
  TensorMaps tm;
  const int group = Hq / Hkv;
  const bool group_fits = group <= kPrefillRows && (kPrefillRows % group) == 0;
  sa.tile_pf = prefill_tile_keys(D);
  sa.pf_min_rows = packed ? packed_prefill_min_rows(sp) : kPrefillRows;
  sa.pf_tile_rows = kTilePrefillRows;
  sa.pf_min_work = packed ? packed_prefill_min_work(sp) : kPrefillMinWork;
  sa.packed = packed != nullptr;
  sa.key_bytes = bits == 8 ? 2 * D : D + D / (kQ4Group / 2);
  sa.sk[0] = sp == PackedSplit::kTile ? tile : few;
  sa.sk[1] = tile;
  sa.sk_choice = sp == PackedSplit::kEither;
  sa.sk_ratio = packed_tile_ratio(bits, D);
  sa.lo_align = packed ? kPackedRows : 1;
  sa.pf_cols = sg.pf_cols;
  // (a call-wide window bounds the positions that a staged column has to hold)
  sa.rows_pf = packed && window > 0 && !sa.seg_mode ? std::min<int64_t>(rows, T + window - 1) : rows;
  sa.prefill_ok = (!packed || sg.pf_cols > 0) && di.prefill_ok[d_index(D)] && group_fits && prefill_launch(sa, T) &&
                  make_tensor_maps(q, T, Hq, D, q_rs, q_hs, packed ? sg.k : k, packed ? sg.v : v, sa.rows_pf,
                                   packed ? sg.pf_cols : cols, Hkv, group, sa.tile_pf, packed != nullptr, &tm.q, &tm.k, &tm.v);
  if (!sa.prefill_ok) sa.pf_cols = 0;
  sa.grid[0] = 0;
  sa.grid[2] = g.prefill;
  sa.ws = W;
  sa.status_dev = status_dev;

  AttnArgs aa{};
  aa.q = (const __nv_bfloat16*)q;
  aa.q_rs = q_rs;
  aa.q_hs = q_hs;
  aa.k = (const __nv_bfloat16*)k;
  aa.v = (const __nv_bfloat16*)v;
  aa.rows = rows;
  aa.cols = cols;
  aa.Hkv = Hkv;
  aa.Hq = Hq;
  aa.group = Hq / Hkv;
  aa.D = D;
  aa.causal = sa.causal;
  aa.window = window;
  aa.scale_log2 = scale * 1.4426950408889634f;
  // (the kernels over codes scale after they mask: a scale of 0 must leave -infinity what it is)
  if (packed) aa.scale_log2 = std::max(aa.scale_log2, FLT_MIN);
  aa.out = (__nv_bfloat16*)out;
  aa.o_rs = o_rs;
  aa.o_hs = o_hs;
  aa.T = T;
  aa.ws = W;
  aa.status_dev = status_dev;
  aa.out_mul = bits == 8 ? kQ8StagedMul : 1.f;
  AppendArgs apw;
  if (ap) {
    apw = *ap;
    apw.segs = W.segs;
  }
  if (bits == 4) packed->q4 = {aa, packed->st, sa.sk_choice};
  if (bits == 8) {
    packed->q8.a = aa;
    packed->q8.st = packed->st;
    packed->q8.choice = sa.sk_choice;
    if (!make_q8_maps(packed->st, rows, cols, Hkv, D, &packed->q8))
      return fail(SDPA_ERR_CUDA, "the 8-bit store's tensor maps could not be made");
  }
  if (parts > 0) {
    const int32_t* table = S > 0 ? seq_info : nullptr;
    PackedDirectArgs<Q4AttnArgs> d4{packed->q4, table, sa.seg_mode, S};
    PackedDirectArgs<Q8AttnArgs> d8{packed->q8, table, sa.seg_mode, S};
    void* args[] = {bits == 8 ? (void*)&d8 : (void*)&d4};
    const cudaStream_t cs = (cudaStream_t)stream;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(T * Hkv * parts));
    cfg.blockDim = dim3(kPackedThreads);
    cfg.dynamicSmemBytes = packed_smem_bytes(bits, D);
    cfg.stream = cs;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)parts;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = mark(i, cs);
    if (e == cudaSuccess) e = cudaLaunchKernelExC(&cfg, packed_direct_ptr(bits, D), args);
    for (int i = 3; i < 5 && e == cudaSuccess; ++i) e = mark(i, cs);
    if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "%d-bit direct launch: %s", bits, cudaGetErrorString(e));
    return SDPA_OK;
  }
  if (sa.pf_cols > 0) {
    sg.segs = W.segs;
    sg.S = S;
    sg.Hkv = Hkv;
    sg.D = D;
    sg.rows = rows;
    sg.rows_pf = sa.rows_pf;
    sg.st = packed->st;
  }
  return launch_all(sa, aa, D, g, tm, ap ? &apw : nullptr, packed, sa.pf_cols > 0 ? &sg : nullptr, (cudaStream_t)stream);
}

// Bytes of workspace of a call over a store of codes; 0 for sizes that it does not take.
static size_t packed_workspace_bytes(int bits, int64_t T, int Hq, int Hkv, int D, int S, int64_t rows, int cols) {
  if (T < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || rows <= 0 || rows > INT32_MAX || cols <= 0) return 0;
  if (D != 64 && D != 128 && D != 256) return 0;
  DevInfo di;
  Grids g{4096, 1024};  // without a device: bounds above any real grid
  SkShape tile{kPackedTileRows, kPackedTileKeys, kSkQ4Tile, 1024};
  if (device_info(&di) == SDPA_OK) {
    g = {packed_resident(di, bits, D), grids_for(di, D).prefill};
    tile = packed_tile_shape(di);
  } else {
    g_err[0] = 0;
  }
  return layout_workspace(nullptr, T, Hq, Hkv, D, S, g.splitk, g.prefill, nullptr, true,
                          D <= 128 ? &tile : nullptr) +
         2 * stage_bytes_per_column(rows, Hkv, D) * packed_stage_cols(bits, T, Hq, Hkv, D, S, rows);
}

static sdpa_status run_packed(int bits, const PackedStore& store, const void* q, int64_t T, int Hq, int D, int64_t q_rs,
                              int64_t q_hs, int64_t rows, int cols, int Hkv, const int32_t* seq_info,
                              const int32_t* seg_mode, int S, int causal, int window, float scale, void* out,
                              int64_t o_rs, int64_t o_hs, void* ws, size_t ws_bytes, int32_t* status_dev,
                              void* stream) {
  // the running maximum is taken over unscaled scores
  if (scale < 0.f) return fail(SDPA_ERR_ARG, "scale %g < 0", (double)scale);
  PackedCall call{};
  call.bits = bits;
  call.st = store;
  return run(q, T, Hq, D, q_rs, q_hs, store.kc, store.vc, rows, cols, Hkv, seq_info, S, nullptr, causal, window, scale,
             out, o_rs, o_hs, ws, ws_bytes, status_dev, stream, nullptr, seg_mode, &call);
}

}  // namespace sdpa

using namespace sdpa;

extern "C" {

size_t sdpa_varlen_workspace_bytes(int64_t T, int Hq, int Hkv, int D, int S) {
  if (T < 0 || S < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return 0;
  if (D != 64 && D != 128 && D != 256) return 0;
  DevInfo di;
  Grids g;
  if (device_info(&di) == SDPA_OK) {
    g = grids_for(di, D);
  } else {
    g.splitk = 4096;  // no device: a bound above any real grid
    g.prefill = 1024;
    g_err[0] = 0;
  }
  return layout_workspace(nullptr, T, Hq, Hkv, D, S, g.splitk, g.prefill, nullptr);
}

sdpa_status sdpa_varlen(const void* q, int64_t T, int Hq, int D, int64_t q_row_stride,
                        int64_t q_head_stride, const void* k_store, const void* v_store,
                        int64_t rows, int cols, int Hkv, const int32_t* seq_info, int S,
                        int causal, int window, float scale, void* out, int64_t o_row_stride,
                        int64_t o_head_stride, void* workspace, size_t ws_bytes,
                        int32_t* status_dev, void* stream) {
  return run(q, T, Hq, D, q_row_stride, q_head_stride, k_store, v_store, rows, cols, Hkv, seq_info,
             S, nullptr, causal, window, scale, out, o_row_stride, o_head_stride, workspace,
             ws_bytes, status_dev, stream);
}

sdpa_status sdpa_varlen_append(const void* q, int64_t T, int Hq, int D, int64_t q_row_stride,
                               int64_t q_head_stride, const void* k_new, const void* v_new,
                               int64_t new_row_stride, int64_t new_head_stride, void* k_store,
                               void* v_store, int64_t rows, int cols, int Hkv, const int32_t* seq_info,
                               int S, int causal, int window, float scale, void* out,
                               int64_t o_row_stride, int64_t o_head_stride, void* workspace,
                               size_t ws_bytes, int32_t* status_dev, void* stream) {
  g_err[0] = 0;
  if (!k_new || !v_new) return fail(SDPA_ERR_NULL, "k_new or v_new is NULL");
  if (!aligned16(k_new) || !aligned16(v_new)) return fail(SDPA_ERR_ALIGN, "k_new and v_new must be 16-byte aligned");
  if (new_row_stride < 0 || new_head_stride < 0 || (new_row_stride % 8) || (new_head_stride % 8))
    return fail(SDPA_ERR_STRIDE, "new-row strides must be non-negative multiples of 8 elements");
  AppendArgs ap{};
  ap.k_new = (const __nv_bfloat16*)k_new;
  ap.v_new = (const __nv_bfloat16*)v_new;
  ap.new_rs = new_row_stride;
  ap.new_hs = new_head_stride;
  ap.k_store = (__nv_bfloat16*)k_store;
  ap.v_store = (__nv_bfloat16*)v_store;
  ap.rows = rows;
  ap.cols = cols;
  ap.Hkv = Hkv;
  ap.D = D;
  return run(q, T, Hq, D, q_row_stride, q_head_stride, k_store, v_store, rows, cols, Hkv, seq_info,
             S, nullptr, causal, window, scale, out, o_row_stride, o_head_stride, workspace,
             ws_bytes, status_dev, stream, &ap);
}

sdpa_status sdpa_varlen_modes(const void* q, int64_t T, int Hq, int D, int64_t q_row_stride,
                              int64_t q_head_stride, const void* k_store, const void* v_store,
                              int64_t rows, int cols, int Hkv, const int32_t* seq_info,
                              const int32_t* seg_mode, int S, float scale, void* out,
                              int64_t o_row_stride, int64_t o_head_stride, void* workspace,
                              size_t ws_bytes, int32_t* status_dev, void* stream) {
  g_err[0] = 0;
  if (!seg_mode && S > 0) return fail(SDPA_ERR_NULL, "seg_mode is NULL");
  return run(q, T, Hq, D, q_row_stride, q_head_stride, k_store, v_store, rows, cols, Hkv, seq_info,
             S, nullptr, 1, 0, scale, out, o_row_stride, o_head_stride, workspace, ws_bytes,
             status_dev, stream, nullptr, seg_mode);
}

size_t sdpa_varlen_fourbit_workspace_bytes(int64_t T, int Hq, int Hkv, int D, int S, int64_t rows, int cols) {
  return packed_workspace_bytes(4, T, Hq, Hkv, D, S, rows, cols);
}

sdpa_status sdpa_varlen_fourbit(const void* q, int64_t T, int Hq, int D, int64_t q_row_stride, int64_t q_head_stride,
                           const sdpa_q4_store* store, int64_t rows, int cols, int Hkv, const int32_t* seq_info,
                           const int32_t* seg_mode, int S, int causal, int window, float scale, void* out,
                           int64_t o_row_stride, int64_t o_head_stride, void* workspace, size_t ws_bytes,
                           int32_t* status_dev, void* stream) {
  g_err[0] = 0;
  if (!store) return fail(SDPA_ERR_NULL, "store is NULL");
  return run_packed(4, {store->k_codes, store->k_scales, store->v_codes, store->v_scales}, q, T, Hq, D, q_row_stride,
                    q_head_stride, rows, cols, Hkv, seq_info, seg_mode, S, causal, window, scale, out, o_row_stride,
                    o_head_stride, workspace, ws_bytes, status_dev, stream);
}

size_t sdpa_varlen_eightbit_workspace_bytes(int64_t T, int Hq, int Hkv, int D, int S, int64_t rows, int cols) {
  return packed_workspace_bytes(8, T, Hq, Hkv, D, S, rows, cols);
}

sdpa_status sdpa_varlen_eightbit(const void* q, int64_t T, int Hq, int D, int64_t q_row_stride, int64_t q_head_stride,
                            const sdpa_q8_store* store, int64_t rows, int cols, int Hkv, const int32_t* seq_info,
                            const int32_t* seg_mode, int S, int causal, int window, float scale, void* out,
                            int64_t o_row_stride, int64_t o_head_stride, void* workspace, size_t ws_bytes,
                            int32_t* status_dev, void* stream) {
  g_err[0] = 0;
  if (!store) return fail(SDPA_ERR_NULL, "store is NULL");
  return run_packed(8, {store->k_codes, store->k_scales, store->v_codes, store->v_scales}, q, T, Hq, D, q_row_stride,
                    q_head_stride, rows, cols, Hkv, seq_info, seg_mode, S, causal, window, scale, out, o_row_stride,
                    o_head_stride, workspace, ws_bytes, status_dev, stream);
}

sdpa_status sdpa_seq_clone(void* k_store, void* v_store, int64_t rows, int cols, int Hkv, int D,
                           int src_col, int dst_col, int64_t n, void* stream) {
  g_err[0] = 0;
  if (!k_store || !v_store) return fail(SDPA_ERR_NULL, "a store pointer is NULL");
  if (!aligned16(k_store) || !aligned16(v_store)) return fail(SDPA_ERR_ALIGN, "stores must be 16-byte aligned");
  if (rows <= 0 || cols <= 0 || Hkv <= 0 || n < 0)
    return fail(SDPA_ERR_SHAPE, "bad sizes: rows=%lld cols=%d Hkv=%d n=%lld", (long long)rows, cols, Hkv,
                (long long)n);
  if (D != 64 && D != 128 && D != 256) return fail(SDPA_ERR_HEAD_DIM, "head dim %d not in {64,128,256}", D);
  if (src_col < 0 || src_col >= cols || dst_col < 0 || dst_col >= cols)
    return fail(SDPA_ERR_ARG, "columns %d -> %d outside [0, %d)", src_col, dst_col, cols);
  const int64_t m = std::min(n, rows);
  if (m == 0 || src_col == dst_col) return SDPA_OK;
  DevInfo di;
  sdpa_status st = device_info(&di);
  if (st) return st;
  CloneArgs ca{};
  ca.k_store = (__nv_bfloat16*)k_store;
  ca.v_store = (__nv_bfloat16*)v_store;
  ca.m = m;
  ca.cols = cols;
  ca.Hkv = Hkv;
  ca.D = D;
  ca.src_col = src_col;
  ca.dst_col = dst_col;
  const int64_t total = m * Hkv * (D / 8);
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((int64_t)di.sms * 8, (total + 4 * kCloneThreads - 1) / (4 * kCloneThreads)));
  void* args[] = {(void*)&ca};
  cudaError_t e = cudaLaunchKernel(clone_kernel_ptr(), dim3((unsigned)blocks), dim3(kCloneThreads), args, 0,
                                   (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "clone launch: %s", cudaGetErrorString(e));
  return SDPA_OK;
}

sdpa_status sdpa_causal_prefill(const void* q, const void* k, const void* v, int64_t Lq,
                                int64_t Lkv, int Hq, int Hkv, int D, float scale, void* out,
                                void* workspace, size_t ws_bytes, void* stream) {
  g_err[0] = 0;
  if (Lq < 0 || Lkv <= 0) return fail(SDPA_ERR_SHAPE, "Lq=%lld Lkv=%lld", (long long)Lq, (long long)Lkv);
  if (Lq > INT32_MAX || Lkv > INT32_MAX) return fail(SDPA_ERR_SHAPE, "Lq or Lkv beyond 2^31-1");
  const int32_t seg[4] = {0, (int32_t)Lq, 0, (int32_t)Lkv};
  const int64_t rs = (int64_t)Hq * D;
  return run(q, Lq, Hq, D, rs, D, k, v, Lkv, 1, Hkv, nullptr, 1, seg, 1, 0, scale, out, rs, D,
             workspace, ws_bytes, nullptr, stream);
}

int sdpa_prefill_available(int D) {
  g_err[0] = 0;
  if (D != 64 && D != 128 && D != 256) {
    fail(SDPA_ERR_HEAD_DIM, "head dim %d not in {64,128,256}", D);
    return -1;
  }
  DevInfo di;
  if (device_info(&di) != SDPA_OK) return -1;
  return di.prefill_ok[d_index(D)] ? 1 : 0;
}

sdpa_status sdpa_set_route_policy(int policy) {
  if (policy != SDPA_ROUTE_AUTO && policy != SDPA_ROUTE_SPLITK && policy != SDPA_ROUTE_PREFILL)
    return fail(SDPA_ERR_ARG, "unknown route policy %d", policy);
  g_policy.store(policy);
  return SDPA_OK;
}

sdpa_status sdpa_set_timing_events(void* const* events, int n) {
  if (!events) {
    g_ev_on = false;
    return SDPA_OK;
  }
  if (n != 5) return fail(SDPA_ERR_ARG, "timing hook takes 5 events, got %d", n);
  for (int i = 0; i < 5; ++i) {
    if (!events[i]) return fail(SDPA_ERR_NULL, "timing event %d is NULL", i);
    g_ev[i] = (cudaEvent_t)events[i];
  }
  g_ev_on = true;
  return SDPA_OK;
}

sdpa_status sdpa_workspace_status(const void* workspace, size_t ws_bytes, int32_t* status_host, void* stream) {
  g_err[0] = 0;
  if (!workspace || !status_host) return fail(SDPA_ERR_NULL, "workspace or status_host is NULL");
  if ((uintptr_t)workspace % 256) return fail(SDPA_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (ws_bytes < sizeof(SchedHdr)) return fail(SDPA_ERR_WORKSPACE, "workspace of %zu bytes has no header", ws_bytes);
  // the header opens every workspace layout; its status word is rewritten by each call's
  // scheduler and ORed by the attention kernels (SDPA_DEV_TIMEOUT)
  const SchedHdr* h = reinterpret_cast<const SchedHdr*>(workspace);
  int64_t v = 0;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(&v, &h->status, sizeof(v), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return fail(SDPA_ERR_CUDA, "status read-back: %s", cudaGetErrorString(e));
  *status_host = (int32_t)v;
  return SDPA_OK;
}

const char* sdpa_last_error(void) { return g_err; }

int sdpa_version(void) { return 100; }

}  // extern "C"
