// q4_attn.cu - split-K attention over the 4-bit column store.
//
// The mathematics of the bf16 split-K kernel (online softmax in base 2 over a CTA's share of a
// unit's keys, partial results joined by log-sum-exp) on keys and values that are turned from
// 4-bit codes into matrix operands in registers.
//
// What bounds it.  A key of one KV head is D codes of K and of V with their scales: 136 bytes at
// D = 128 against 512 in bf16.  At the measured copy rate that is one key per 5.8 SM cycles, and
// each brings 256 values to convert, so the instructions that convert (11 to 12 per 8 values, see
// q4.cuh) weigh as much as the loads.  Everything else is therefore kept off the issue slots:
//   * a fifth warp loads: whole runs of store rows by bulk copies (one thread, four copies per
//     stage) into a ring of stages, across the borders of pieces, so that the next piece's first
//     keys (and its query rows) travel while this one is finished;
//   * no value is written back to shared memory: codes are read once per warp, as whole words, in
//     an order that makes them operand fragments at once.  The contraction over dims does not care
//     about their order, so a lane of K takes D / 4 dims of its key side by side (with their one
//     or two scales), and the query fragments follow; a lane of V takes D / 8 dims side by side of
//     four keys, and the output's rows follow;
//   * scales are multiplied in by the conversion's own fused multiply-add, exactly;
//   * the products are taken transposed, S^T = K Q^T and O^T = V^T P^T: keys and dims fill the
//     16 rows of an m16n8k16 product and the query rows its 8 columns, so that a decode unit of up
//     to 8 rows (one token's heads) wastes no half of each product, score and output register.
//     P^T is the transpose of what S^T leaves in the lanes: one movmatrix per 8 x 8 block.
//     (With the query rows as the 16 rows a decode of 64 sequences over 24576 keys on average, 8 KV
//     heads, D = 128, took 675 us, and 466 so; 335 us, 5.2 TB/s of codes and scales, with what
//     follows.  No pipe is full then: the ALU pipe is busy 55 % of the time, at 2.3 of 4 instructions a
//     cycle, and the 10 warps of an SM wait for their own results (0.7 cycles an instruction) and loads
//     (0.7).  A third CTA on an SM, with runs of 32 keys to fit its registers, took 356 us.)
// P is rounded to fp16 (half a step is at most 2^-11 of it, against 2^-8 in bf16) and V is exact in
// fp16; Q and K are multiplied in bf16, where both are exact.  Sums are fp32.  The lazily updated
// maximum leaves P at most 2^8 above it, so P is kept 2^7 times larger, its sum too: at most 2^15,
// and a row's largest at least 2^7, so that a P that fp16's smallest step (2^-24) cannot hold is
// less than 2^-32 of its row: a million such keys are still lost in the output's rounding.
#include "packed_attn.cuh"
#include "q4.cuh"

namespace sdpa {

// A unit of more than 8 rows is converted again for every 8 of them.  (16 rows a warp, twice the registers
// of output, made a CTA of 168 registers and units of 8 rows slower by a tenth; segments of more than 16
// rows have a kernel of their own, q4_tile.cu.)
template <int D>
struct Q4Few {
  using Args = Q4AttnArgs;
  static constexpr int kRun = D == 256 ? 2 : 4;  // 16-key blocks between two looks at the maximum
  static constexpr int kKeys = 64 * kRun;        // keys per stage of the ring
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kPerSm = D == 64 ? 3 : 2;  // CTAs per SM that registers and shared memory allow
  static constexpr int kRowBytes = D / 2;
  static constexpr int kScaleBytes = D / kQ4Group;
  static constexpr int kCodes = kKeys * kRowBytes;
  static constexpr int kScales = kKeys * kScaleBytes;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kQPitch = D * 2 + 16;
  static constexpr int kQBytes = kSplitkRows * kQPitch;
  static constexpr int kMerge = 8;
  static constexpr int kMergeBytes = 4 * 8 * 68 * 4;  // 64 dims of the warps' rows
  static constexpr int kBytes = kRingBytes + kQBytes + kMergeBytes;
  static constexpr SkKind kKind = kSkQ4Few;
  static constexpr int kAlign = 16, kFull = 1;
  static constexpr float kOut = 1.f;
  static constexpr int WK = D / 32;  // words of a lane's K chunk (D / 4 dims)
  static constexpr int WV = D / 64;  // words of a lane's V chunk (D / 8 dims)

  __device__ __forceinline__ static const char* side(const char* ring, uint32_t st) {
    return ring + st * kStageBytes + 2 * kCodes;
  }

  // The keys of a stage span at most rows + 15 positions from a multiple of 16 on, so they are at most two runs of
  // store rows, both of whole 16-row blocks.
  struct Loader {
    const Q4AttnArgs& G;
    const int64_t plane;  // first row of the column's head
    const int lane;
    __device__ __forceinline__ Loader(const Q4AttnArgs& g, const UnitRec& ur, int l)
        : G(g), plane(((int64_t)ur.col * g.a.Hkv + ur.hk) * g.a.rows), lane(l) {}
    __device__ __forceinline__ void start(int64_t, int) {}
    __device__ __forceinline__ void stage(char* ring, uint32_t st, uint32_t bar, int64_t row, int rows16) {
      if (lane != 0) return;
      const int first = (int)min((int64_t)rows16, G.a.rows - row), second = rows16 - first;
      const uint32_t dst = smem_u32(ring + st * kStageBytes);
      mbar_expect_tx(bar, (uint32_t)rows16 * 2 * (kRowBytes + kScaleBytes));
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint8_t* codes = v ? G.st.vc : G.st.kc;
        const uint8_t* scales = v ? G.st.vs : G.st.ks;
        const uint32_t dc = dst + v * kCodes, ds = dst + 2 * kCodes + v * kScales;
        bulk_load(dc, codes + (plane + row) * kRowBytes, first * kRowBytes, bar);
        bulk_load(ds, scales + (plane + row) * kScaleBytes, first * kScaleBytes, bar);
        if (second > 0) {
          bulk_load(dc + first * kRowBytes, codes + plane * kRowBytes, second * kRowBytes, bar);
          bulk_load(ds + first * kScaleBytes, scales + plane * kScaleBytes, second * kScaleBytes, bar);
        }
      }
    }
  };

  struct Query {
    uint4 f[WK];
    const float sl2;
    __device__ __forceinline__ Query(const char* row, int tq, float scale_log2) : sl2(scale_log2) {
      const char* qrow = row + tq * (D / 2);
#pragma unroll
      for (int w = 0; w < WK; ++w) f[w] = q4_q_order(*reinterpret_cast<const uint4*>(qrow + 16 * w));
    }
    __device__ __forceinline__ float scale(int) const { return sl2; }
  };

  // Row n of 8 keys stands for key n, with the two of every other pair swapped: the four lanes of a
  // quad then read V rows of both parities (rows of one parity share banks).
  struct Operands {
    const uint32_t kbits, vbits;
    const int gq, tq;
    const int kn;  // the key of this lane's K row
    const int ko;  // the keys of its V columns: ko and ko ^ 1
    __device__ __forceinline__ Operands(int lane)
        : kbits(in_register(kQ4Bf16)), vbits(in_register(kQ4F16)), gq(lane >> 2), tq(lane & 3),
          kn(gq ^ ((gq >> 1) & 1)), ko(2 * tq + (tq & 1)) {}

    __device__ __forceinline__ void scores(const char* kc, const char* ks, int key0, const Query& q,
                                           float (&s)[4]) const {
      const int key = key0 + kn;
      uint32_t kw[2][WK];  // keys key and key + 8
      __nv_bfloat162 s2[2], z2[2];
      const uint8_t* sb = reinterpret_cast<const uint8_t*>(ks) + key * kScaleBytes + tq * D / 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lds_words<WK>(kc + (key + 8 * h) * kRowBytes + tq * (D / 8), kw[h]);
        q4_scales_bf16(sb[8 * h * kScaleBytes], &s2[h], &z2[h]);
      }
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        if constexpr (D == 256) {
          if (w == 4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) q4_scales_bf16(sb[8 * h * kScaleBytes + 1], &s2[h], &z2[h]);
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // two k-steps of 16 dims
          uint32_t a[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[2 * i] = q4_pair_bf16(kw[0][w] >> (8 * x + 4 * i), kbits, s2[0], z2[0]);
            a[2 * i + 1] = q4_pair_bf16(kw[1][w] >> (8 * x + 4 * i), kbits, s2[1], z2[1]);
          }
          mma_bf16_16816(s, a, x ? q.f[w].z : q.f[w].x, x ? q.f[w].w : q.f[w].y);
        }
      }
    }

    __device__ __forceinline__ void values(const char* stage, const char* side, int key0, uint32_t b0, uint32_t b1,
                                           float (&o)[D / 16][4]) const {
      const char* vc = stage + kCodes;
      const char* vs = side + kScales;
      uint32_t vw[4][WV];  // keys ko, ko ^ 1 of the first 8, then of the second
      uint32_t sb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = key0 + 8 * (e >> 1) + (ko ^ (e & 1));
        lds_words<WV>(vc + k * kRowBytes + gq * (D / 16), vw[e]);
        sb[e] = reinterpret_cast<const uint8_t*>(vs)[k * kScaleBytes + gq * D / 256];
      }
      __half2 s2[2], z2[2];
      q4_scales_f16(sb[0], sb[1], &s2[0], &z2[0]);
      q4_scales_f16(sb[2], sb[3], &s2[1], &z2[1]);
#pragma unroll
      for (int w = 0; w < WV; ++w) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // low and high halves: dims 8w .. 8w + 3, 8w + 4 .. 8w + 7
          const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], hf ? 0x7632 : 0x5410);
          const uint32_t x1 = __byte_perm(vw[2][w], vw[3][w], hf ? 0x7632 : 0x5410);
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            uint32_t a[4];
            a[0] = q4_pair_f16(i == 0 ? x0 << 6 : x0 >> 2, vbits, s2[0], z2[0]);
            a[1] = q4_pair_f16(i == 0 ? x0 << 2 : x0 >> 6, vbits, s2[0], z2[0]);
            a[2] = q4_pair_f16(i == 0 ? x1 << 6 : x1 >> 2, vbits, s2[1], z2[1]);
            a[3] = q4_pair_f16(i == 0 ? x1 << 2 : x1 >> 6, vbits, s2[1], z2[1]);
            mma_f16_16816(o[4 * w + 2 * hf + i / 2], a, b0, b1);
          }
        }
      }
    }
  };
};

template <int D>
__global__ void __launch_bounds__(kPackedThreads, Q4Few<D>::kPerSm) sdpa_q4_splitk_kernel(Q4AttnArgs G) {
  extern __shared__ __align__(128) char smem[];
  packed_splitk<D, Q4Few<D>>(G, smem);
}
template <int D>
__global__ void __launch_bounds__(kPackedThreads, Q4Few<D>::kPerSm)
    sdpa_q4_direct_kernel(PackedDirectArgs<Q4AttnArgs> G) {
  extern __shared__ __align__(128) char smem[];
  packed_direct<D, Q4Few<D>>(G, smem);
}

template __global__ void sdpa_q4_splitk_kernel<64>(Q4AttnArgs);
template __global__ void sdpa_q4_splitk_kernel<128>(Q4AttnArgs);
template __global__ void sdpa_q4_splitk_kernel<256>(Q4AttnArgs);

int q4_splitk_smem_bytes(int D) {
  switch (D) {
    case 64: return Q4Few<64>::kBytes;
    case 128: return Q4Few<128>::kBytes;
    default: return Q4Few<256>::kBytes;
  }
}

const void* q4_splitk_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q4_splitk_kernel<64>;
    case 128: return (const void*)sdpa_q4_splitk_kernel<128>;
    default: return (const void*)sdpa_q4_splitk_kernel<256>;
  }
}

const void* q4_direct_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q4_direct_kernel<64>;
    case 128: return (const void*)sdpa_q4_direct_kernel<128>;
    default: return (const void*)sdpa_q4_direct_kernel<256>;
  }
}

}  // namespace sdpa
