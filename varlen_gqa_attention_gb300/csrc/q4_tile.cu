// q4_tile.cu - attention over the 4-bit column store for segments of several rows (draft blocks, short
// chunks), on the tensor-memory tensor cores; D = 64 and 128.
//
// The split-K kernel of q4_attn.cu turns every key into operands once for 8 query rows; a block of 16
// draft rows with 4 heads a KV head is 64, and converting is what that kernel does most.  Here a key is
// converted once for up to 128 rows: S = Q K^T (128 rows x 128 keys) and O += P V are tcgen05 products, Q,
// K and V in shared memory, S, P and O in tensor memory.  Per CTA (one per SM), 18 warps:
//   * a loading warp walks the CTA's pieces (the split-K route's, in units of 128 packed rows and tiles of
//     128 keys), hands them on, and streams their codes and scales into a ring by bulk copies;
//   * eight converting warps, four for every other tile, turn a tile's codes into bf16 K and fp16 V tiles
//     (exactly: see q4.cuh), written in the 128-byte swizzle that the products read; all eight bring a
//     piece's query rows there;
//   * one warp issues the products: S(0) S(1) | PV(0) S(2) | PV(1) S(3) ...  P lies over the scores it came
//     from, which the next scores of that buffer overwrite behind PV (one thread's products run in order);
//   * eight softmax warps, four for a tile's first 64 keys and four for the others.  The two halves keep
//     maxima, sums and an output of their own, as if they were two CTAs' pieces, and are joined when the
//     piece ends: nothing passes between them in between.  A warp can reach the tensor-memory lanes of one
//     quarter only, so a unit of up to 64 rows has 16 of them in each quarter (8, when 32 are all), and the
//     four threads of a quad share a row; a larger unit has a thread a row.
// A word of codes gives its values in pairs (dim i, dim i + 4); K and V tiles keep that order, and so do
// the query rows, and the output's columns are put in order as they are written.
// P is fp16, held 2^7 times larger, as in q4_attn.cu.
//
// Bound by latency: a tile of 64 rows at D = 128 is about six thousand instructions (conversion two of them), issued
// at 1.7 of 4 a cycle, while the tensor cores are busy a third of the time and shared memory two fifths.  The
// softmax warps wait for each tensor-memory load and store in the statement that issues it (long scoreboard
// 3.5 cycles an instruction), and 576 threads leave 96 registers each, which spill (52 bytes at D = 128, 32
// at 64).  64 segments over 6144 keys on average, 8 KV heads, D = 128: 24 rows 150 us, 64
// rows 158 us.  With the rows packed (the softmax of 32 rows all in one quarter, on one scheduler) and four
// converting warps: 221 and 205 us.  (Products of 64 rows instead of 128, and codes read without bank
// conflicts, came to the same; so did rows copied to every quarter, each with its share of the keys, and one
// team converting K and the other V.  Softmax teams that take whole tiles in turn: 203 us for 64 rows: the chain
// scores - probabilities - product of a tile is then longer, and two tiles in flight do not hide it.)
#include "packed_tile.cuh"
#include "q4.cuh"

namespace sdpa {

template <int D>
struct Q4Tile {
  using Args = Q4AttnArgs;
  static constexpr int kRowBytes = D / 2;
  static constexpr int kScaleBytes = D / kQ4Group;
  static constexpr int kKeys = kPackedTileKeys;
  static constexpr int kCodes = kKeys * kRowBytes;
  static constexpr int kScales = kKeys * kScaleBytes;
  static constexpr int kCodeBytes = 2 * (kCodes + kScales);
  static constexpr int kCodeStages = 3;
  static constexpr int kTileBytes = 128 * D * 2;  // Q, or K or V of one stage
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kTileBytes;  // two stages
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffCodes = kOffV + 2 * kTileBytes;
  // (at D = 64 too, more than half of an SM's: a second CTA would only wait for tensor memory)
  static constexpr int kUsed = kOffCodes + kCodeStages * kCodeBytes + 1024;  // + alignment slack
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  // tensor memory columns: S_b fp32 (P_b as fp16 pairs over the first 32 of each half's 64), O of each half
  static constexpr int kColS = 0;
  static constexpr int kColO = 256;
  static constexpr int kParts = 1, kFull = 1;
  static constexpr bool kPairs = true;
  static constexpr SkKind kKind = kSkQ4Tile;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
  static constexpr float kOut = 1.f;
  static constexpr int NH = D / 64;  // 64-dim columns of the tile

  // A tile is at most two runs of store rows, both of whole 16-row blocks (a piece begins at a multiple of 16, a
  // unit spans at most rows + 15 positions).
  struct Loader {
    const Q4AttnArgs& G;
    const int64_t plane;  // first row of the column's head
    const int lane;
    __device__ __forceinline__ Loader(const Q4AttnArgs& g, const UnitRec& ur, int l)
        : G(g), plane(((int64_t)ur.col * g.a.Hkv + ur.hk) * g.a.rows), lane(l) {}
    __device__ __forceinline__ void start(int64_t, int) {}
    __device__ __forceinline__ void stage(uint8_t* smem, uint32_t st, uint32_t bar, int, int64_t row, int rows16) {
      if (lane != 0) return;
      const int first = (int)min((int64_t)rows16, G.a.rows - row), second = rows16 - first;
      const uint32_t dst = smem_u32(smem) + kOffCodes + st * kCodeBytes;
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

  struct Codes {
    uint4 w[2][2][NH];  // [K, V][key0, key0 + 64]
    uint32_t sb[2][2][NH];
  };
  struct Convert {
    const uint32_t kbits, vbits;
    __device__ __forceinline__ explicit Convert(int) : kbits(in_register(kQ4Bf16)), vbits(in_register(kQ4F16)) {}
    __device__ __forceinline__ void read(const uint8_t* smem, uint32_t st, int, int key0, int half, Codes& x) const {
      const uint8_t* codes = smem + kOffCodes + st * kCodeBytes;
      const uint8_t* scales = codes + 2 * kCodes;
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < NH; ++c) {
            const int key = key0 + 64 * i;
            x.w[v][i][c] = *reinterpret_cast<const uint4*>(codes + v * kCodes + key * kRowBytes + c * 32 + half * 16);
            x.sb[v][i][c] = scales[v * kScales + key * kScaleBytes + c * 2 + half];
          }
    }
    __device__ __forceinline__ void keys(const Codes& x, uint8_t* kt, int key0, int half) const {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NH; ++c) {
          __nv_bfloat162 s2, z2;
          q4_scales_bf16(x.sb[0][i][c], &s2, &z2);
          const uint32_t y[4] = {x.w[0][i][c].x, x.w[0][i][c].y, x.w[0][i][c].z, x.w[0][i][c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(kt + c * (128 * 128) + swz(key0 + 64 * i, half * 4 + k, 128)) =
                make_uint4(q4_pair_bf16(y[k], kbits, s2, z2), q4_pair_bf16(y[k] >> 4, kbits, s2, z2),
                           q4_pair_bf16(y[k] >> 8, kbits, s2, z2), q4_pair_bf16(y[k] >> 12, kbits, s2, z2));
        }
    }
    __device__ __forceinline__ void values(const Codes& x, uint8_t* vt, int key0, int half) const {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < NH; ++c) {
          __half2 s2, z2;
          q4_scales_f16(x.sb[1][i][c], x.sb[1][i][c], &s2, &z2);
          const uint32_t y[4] = {x.w[1][i][c].x, x.w[1][i][c].y, x.w[1][i][c].z, x.w[1][i][c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(vt + c * (128 * 128) + swz(key0 + 64 * i, half * 4 + k, 128)) =
                make_uint4(q4_pair_f16(y[k] << 6, vbits, s2, z2), q4_pair_f16(y[k] << 2, vbits, s2, z2),
                           q4_pair_f16(y[k] >> 2, vbits, s2, z2), q4_pair_f16(y[k] >> 6, vbits, s2, z2));
        }
    }
  };

  __device__ __forceinline__ static uint4 query(const uint4& q) { return q4_q_order(q); }
  struct RowScale {
    static constexpr bool kOwn = false;
    __device__ __forceinline__ void set(int, const __nv_bfloat16*, int, int, float) {}
    __device__ __forceinline__ float get(int, float call) const { return call; }
  };
};

template <int D>
__global__ void __launch_bounds__(kPackedTileThreads, 1) sdpa_q4_tile_kernel(Q4AttnArgs G) {
  extern __shared__ uint8_t smem_raw[];
  packed_tile<D, Q4Tile<D>>(G, smem_raw);
}

template __global__ void sdpa_q4_tile_kernel<64>(Q4AttnArgs);
template __global__ void sdpa_q4_tile_kernel<128>(Q4AttnArgs);

const void* q4_tile_kernel_ptr(int D) {
  return D == 64 ? (const void*)sdpa_q4_tile_kernel<64> : (const void*)sdpa_q4_tile_kernel<128>;
}
int q4_tile_smem_bytes(int D) { return D == 64 ? Q4Tile<64>::kBytes : Q4Tile<128>::kBytes; }

}  // namespace sdpa
