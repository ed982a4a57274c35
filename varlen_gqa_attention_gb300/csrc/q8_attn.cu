// q8_attn.cu - attention of few rows over the 8-bit column store (the kernels of packed_attn.cuh).
//
// What bounds it: a key of one KV head is D bytes of K and of V and an eighth of a byte of scales, at the measured
// copy rate one key per 11 SM cycles at D = 128; its 256 values take two instructions for every two of them to become
// matrix operands (a byte permutation that puts the code under the exponent of 1024, then one fused
// multiply-add, see q8.cuh), so that converting takes a fifth of the issue slots of that time.
//   * K and V are both multiplied in fp16, of their values / 16: exact, and the fused multiply-add's
//     addend -1152 s / 16 stays finite up to the largest scale.  The factor 16 goes into the scores' scale and the
//     output.
//   * The queries come to fp16 by a power of two for each row, which brings the row's largest magnitude into
//     [2^14, 2^15): what is above 2^-31 of it is exact, what is below is off by at most 2^-39 of it.  The opposite
//     power goes into the scale of the row's scores.
//   * A stage is loaded by TMA, in one box for K and one for V or in boxes of 16 rows at the ends, swizzled so that both
//     the K reads (16 codes of 8 rows) and the V reads (16 codes of 4 rows) of eight lanes meet all banks.  A lane each
//     brings a block's scale byte, fetched while the stage before was waited for, as an fp16 pair.  (Bytes fetched by the
//     attention warps, a stage ahead, took 24.3 us for the 32 tokens below, 22.6 so.)
// Measured (one GB300, in a graph): 64 tokens over 16384 to 32768 keys, 32/8 heads, D = 128: 490 to 493 us, 6.7 TB/s of codes and
// scales, the measured copy rate; D = 256 (16/4 heads, 16384 keys each) 6.6 TB/s, D = 64 5.8.  32 tokens over up to 8192
// keys, 16/2 heads, without a schedule: 20.1 us, 22.4 over cold keys.  The longest range alone among ranges of 16 keys takes
// 17.9 (all of 16 keys 7.4): 2048 keys a CTA at 0.66 us for each 128 of them, the latency of their scores,
// probabilities and products in turn.
// P is rounded to fp16 as over the 4-bit store (q4_attn.cu), sums are fp32.
#include "packed_attn.cuh"
#include "q8.cuh"

namespace sdpa {

template <int D>
struct Q8Few {
  using Args = Q8AttnArgs;
  static constexpr int kRun = D == 64 ? 4 : D == 128 ? 2 : 1;  // 16-key blocks between two looks at the maximum
  static constexpr int kKeys = 64 * kRun;
  static constexpr int kStages = D == 128 ? 3 : 2;
  static constexpr int kPerSm = D == 64 ? 3 : 2;  // CTAs per SM that registers and shared memory allow
  static constexpr int kPitch = D == 64 ? 64 : 128;  // bytes of a swizzled row; D = 256 has two planes of them
  static constexpr int kPlanes = D / kPitch, kPlane = kKeys * kPitch;
  static constexpr int kCodes = kKeys * D;
  static constexpr int kBlocks = kKeys / kPackedRows;
  static constexpr int kStageBytes = 2 * kCodes;
  static constexpr int kSideBytes = 2 * kBlocks * 4;  // of K's blocks, then of V's: (s / 16, s / 16) in fp16
  static constexpr int kRingBytes = kStages * (kStageBytes + kSideBytes);
  static constexpr int kQPitch = D * 2 + 16;
  static constexpr int kQBytes = kSplitkRows * kQPitch;
  static constexpr int kMerge = D == 256 ? 16 : 4;  // (what shared memory leaves room for)
  static constexpr int kMergeBytes = 4 * 8 * (8 * kMerge + 4) * 4;
  static constexpr int kAlign = 8 * kPitch, kFull = 2;
  static constexpr int kBytes = kRingBytes + kQBytes + kMergeBytes + kAlign;
  static constexpr SkKind kKind = kSkQ8Few;
  static constexpr float kOut = 16.f;
  static constexpr int NK = D == 64 ? 1 : 2;  // 16-byte chunks of a lane's K row in a plane
  static constexpr int NV = D == 256 ? 2 : 1;  // of its V row (D = 64: half a chunk)

  __device__ __forceinline__ static const char* side(const char* ring, uint32_t st) {
    return ring + kStages * kStageBytes + st * kSideBytes;
  }

  struct Loader {
    const Q8AttnArgs& G;
    const int64_t plane;  // first row of the column's head
    const int col_head, lane, block, value;
    uint32_t byte;
    __device__ __forceinline__ Loader(const Q8AttnArgs& g, const UnitRec& ur, int l)
        : G(g), plane(((int64_t)ur.col * g.a.Hkv + ur.hk) * g.a.rows), col_head(ur.col * g.a.Hkv + ur.hk), lane(l),
          block(l % kBlocks), value(l / kBlocks), byte(0) {}
    __device__ __forceinline__ bool mine(int rows16) const { return value < 2 && block * kPackedRows < rows16; }
    __device__ __forceinline__ int64_t my_row(int64_t row) const {
      const int64_t r = row + block * kPackedRows;
      return r >= G.a.rows ? r - G.a.rows : r;
    }
    __device__ __forceinline__ void start(int64_t row, int rows16) {
      if (mine(rows16)) byte = (value ? G.st.vs : G.st.ks)[(plane + my_row(row)) / kPackedRows];
    }
    __device__ __forceinline__ void stage(char* ring, uint32_t st, uint32_t bar, int64_t row, int rows16) {
      if (lane == 0) mbar_expect_tx(bar, (uint32_t)rows16 * 2 * D);
      __syncwarp();
      uint32_t t = 0;  // of a block that is not loaded: what lies there stays finite
      const uint32_t dst = smem_u32(ring + st * kStageBytes) + value * kCodes;
      if (rows16 == kKeys && row + kKeys <= G.a.rows) {  // the stage in one run of store rows
        if (value < 2 && block == 0) {
          constexpr int kBox = q8_box_rows(D);
#pragma unroll
          for (int i = 0; i < kKeys; i += kBox)
#pragma unroll
            for (int p = 0; p < kPlanes; ++p)
              tma_load_3d(dst + p * kPlane + i * kPitch, value ? &G.v_box : &G.k_box, bar, p * kPitch, (int)row + i, col_head);
        }
      } else if (mine(rows16)) {
#pragma unroll
        for (int p = 0; p < kPlanes; ++p)
          tma_load_3d(dst + p * kPlane + block * (kPackedRows * kPitch), value ? &G.v : &G.k, bar, p * kPitch,
                      (int)my_row(row), col_head);
      }
      if (mine(rows16)) t = q8_scale_f16x2(byte);
      if (value < 2)
        *reinterpret_cast<uint32_t*>(ring + kStages * kStageBytes + st * kSideBytes + (value * kBlocks + block) * 4) =
            t;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    }
  };

  struct Query {
    uint32_t f[D / 8];
    float sl2[2];
    __device__ __forceinline__ Query(const char* row, int tq, float scale_log2) {
      uint4 w[D / 32];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // (a plane's 32 dims of the lane are side by side)
        w[i] = *reinterpret_cast<const uint4*>(row + i / (kPitch / 32) * (2 * kPitch) + tq * (kPitch / 2) +
                                               i % (kPitch / 32) * 16);
        amax = q8_row_amax(w[i], amax);
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const uint32_t up = q8_row_up(amax);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = q8_row_f16(w[i], __uint_as_float(up << 23));
        f[4 * i] = x.x; f[4 * i + 1] = x.y; f[4 * i + 2] = x.z; f[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
        sl2[c] = q8_row_scale(__shfl_sync(0xffffffffu, up, 4 * (2 * tq + c)), scale_log2);
    }
    __device__ __forceinline__ float scale(int c) const { return sl2[c]; }
  };

  // Row n of 8 keys stands for key n, with the two of every other pair swapped: the four lanes of a
  // quad then read V rows of both parities (at D = 64 rows of one parity share banks).
  struct Operands {
    const uint32_t magic;
    const int gq, tq;
    const int kn;  // the key of this lane's K row
    const int ko;  // the keys of its V columns: ko and ko ^ 1
    __device__ __forceinline__ Operands(int lane)
        : magic(in_register(kQ8Magic)), gq(lane >> 2), tq(lane & 3), kn(gq ^ ((gq >> 1) & 1)),
          ko(2 * tq + (tq & 1)) {}

    template <bool HI>
    __device__ __forceinline__ uint32_t pair(uint32_t x, __half2 t, __half2 z) const {
      return q8_pair_f16<HI>(x, magic, t, z);
    }
    __device__ __forceinline__ static void scales(const char* side, int block, __half2* t, __half2* z) {
      *t = *reinterpret_cast<const __half2*>(side + 4 * block);
      *z = __hmul2(*t, __float2half2_rn(-1152.f));
    }

    __device__ __forceinline__ void scores(const char* stage, const char* side, int key0, const Query& q,
                                           float (&s)[4]) const {
      __half2 t, z;
      scales(side, key0 / kPackedRows, &t, &z);
      const char* row = stage + (key0 + kn) * kPitch;
#pragma unroll
      for (int p = 0; p < kPlanes; ++p) {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          const int at = D == 64 ? (tq ^ (kn >> 1 & 3)) << 4 : ((2 * tq + i) ^ kn) << 4;
          const uint4 x = *reinterpret_cast<const uint4*>(row + p * kPlane + at);
          const uint4 y = *reinterpret_cast<const uint4*>(row + p * kPlane + 8 * kPitch + at);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a[4] = {pair<false>(xs[w], t, z), pair<false>(ys[w], t, z), pair<true>(xs[w], t, z),
                                   pair<true>(ys[w], t, z)};
            const int at_q = 2 * ((p * NK + i) * 4 + w);
            mma_f16_16816(s, a, q.f[at_q], q.f[at_q + 1]);
          }
        }
      }
    }

    __device__ __forceinline__ void values(const char* stage, const char* side, int key0, uint32_t b0, uint32_t b1,
                                           float (&o)[D / 16][4]) const {
      __half2 t, z;
      scales(side, kBlocks + key0 / kPackedRows, &t, &z);
      const char* rows = stage + kCodes + (D == 256 ? (gq >> 2) * kPlane : 0) + key0 * kPitch;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        constexpr int NW = D == 64 ? 2 : 4;
        uint32_t v[4][NW];  // keys ko, ko ^ 1 of the first 8, then of the second
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = ko ^ (e & 1);
          const char* row = rows + (8 * (e >> 1) + r) * kPitch;
          if constexpr (D == 64)
            lds_words<NW>(row + (((gq >> 1) ^ (r >> 1 & 3)) << 4) + (gq & 1) * 8, v[e]);
          else
            lds_words<NW>(row + (((D == 256 ? 2 * (gq & 3) + i : gq) ^ r) << 4), v[e]);
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            // (the two keys' codes of a dim side by side, for two dims)
            const uint32_t x = __byte_perm(v[0][w], v[1][w], hf ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(v[2][w], v[3][w], hf ? 0x7362 : 0x5140);
            const uint32_t a[4] = {pair<false>(x, t, z), pair<true>(x, t, z), pair<false>(y, t, z),
                                   pair<true>(y, t, z)};
            mma_f16_16816(o[2 * (i * NW + w) + hf], a, b0, b1);
          }
        }
      }
    }
  };
};

template <int D>
__global__ void __launch_bounds__(kPackedThreads, Q8Few<D>::kPerSm)
    sdpa_q8_splitk_kernel(const __grid_constant__ Q8AttnArgs G) {
  extern __shared__ __align__(128) char smem[];
  packed_splitk<D, Q8Few<D>>(G, smem);
}
template <int D>
__global__ void __launch_bounds__(kPackedThreads, Q8Few<D>::kPerSm)
    sdpa_q8_direct_kernel(const __grid_constant__ PackedDirectArgs<Q8AttnArgs> G) {
  extern __shared__ __align__(128) char smem[];
  packed_direct<D, Q8Few<D>>(G, smem);
}

int q8_splitk_smem_bytes(int D) {
  switch (D) {
    case 64: return Q8Few<64>::kBytes;
    case 128: return Q8Few<128>::kBytes;
    default: return Q8Few<256>::kBytes;
  }
}
const void* q8_splitk_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q8_splitk_kernel<64>;
    case 128: return (const void*)sdpa_q8_splitk_kernel<128>;
    default: return (const void*)sdpa_q8_splitk_kernel<256>;
  }
}
const void* q8_direct_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q8_direct_kernel<64>;
    case 128: return (const void*)sdpa_q8_direct_kernel<128>;
    default: return (const void*)sdpa_q8_direct_kernel<256>;
  }
}

}  // namespace sdpa
