// q8_tile.cu - attention over the 8-bit column store for segments of several rows, on the tensor-memory tensor cores;
// D = 64 and 128.  The kernel is that of packed_tile.cuh (its parts are described in q4_tile.cu).
//
// As in q8_attn.cu both K and V are brought to fp16, of their values / 16, two instructions for two of them, and the
// query rows by a power of two each; the converting warps find a row's power as they bring it into shared memory,
// and the softmax warps find it again for the rows whose scores they scale (a row's loads travel while the first
// tile is made).  K's and V's codes of a tile are stages of their own in the ring (D = 128: 16 KB each, three of them
// beside the tiles), loaded by TMA in swizzled boxes.
//
// Bound by latency as the 4-bit store's (1.4 instructions a cycle, the tensor cores busy a quarter of the time), and at
// D = 128 by the tile and a half that fit the ring: 32 segments of 16 tokens over 8192 keys, 32/8 heads, take 174 us, 157 over
// keys that lie in the L2 (the 4-bit store 148 and 142); 16 segments of 1 to 16 tokens within 4096-key windows 61 us with
// the schedule and joining, 53 here.
#include "packed_tile.cuh"
#include "q8.cuh"

namespace sdpa {

template <int D>
struct Q8Tile {
  using Args = Q8AttnArgs;
  static constexpr int kKeys = kPackedTileKeys;
  static constexpr int kPitch = D;  // bytes of a swizzled row
  static constexpr int kCodeBytes = kKeys * D;
  static constexpr int kBlocks = kKeys / kPackedRows;
  static constexpr int kCodeStages = D == 128 ? 3 : 6;
  static constexpr int kTileBytes = 128 * D * 2;  // Q, or K or V of one stage
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kTileBytes;  // two stages
  static constexpr int kOffV = kOffK + 2 * kTileBytes;
  static constexpr int kOffCodes = kOffV + 2 * kTileBytes;
  static constexpr int kOffScales = kOffCodes + kCodeStages * kCodeBytes;  // (s / 16, s / 16) in fp16, of each block
  // (at D = 64 too, more than half of an SM's: a second CTA would only wait for tensor memory)
  static constexpr int kUsed = kOffScales + kCodeStages * kBlocks * 4 + 1024;  // + alignment slack
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  // tensor memory columns: S_b fp32 (P_b as fp16 pairs over the first 32 of each half's 64), O of each half
  static constexpr int kColS = 0;
  static constexpr int kColO = 256;
  static constexpr int kParts = 2, kFull = 2;
  static constexpr bool kPairs = false;
  static constexpr SkKind kKind = kSkQ4Tile;
  static constexpr uint32_t kIdescS = idesc_f16_f32(128, 128, false, false);
  static constexpr float kOut = 16.f;
  static constexpr int NH = D / 64;  // 64-dim columns of the tile

  struct Loader {
    const Q8AttnArgs& G;
    const int64_t plane;  // first row of the column's head
    const int col_head, lane, block, value;
    uint32_t byte;
    __device__ __forceinline__ Loader(const Q8AttnArgs& g, const UnitRec& ur, int l)
        : G(g), plane(((int64_t)ur.col * g.a.Hkv + ur.hk) * g.a.rows), col_head(ur.col * g.a.Hkv + ur.hk), lane(l),
          block(l % kBlocks), value(l / kBlocks), byte(0) {}
    __device__ __forceinline__ int64_t my_row(int64_t row) const {
      const int64_t r = row + block * kPackedRows;
      return r >= G.a.rows ? r - G.a.rows : r;
    }
    // lanes [0, kBlocks) keep K's bytes, the next ones V's
    __device__ __forceinline__ void start(int64_t row, int rows16) {
      if (value < 2 && block * kPackedRows < rows16)
        byte = (value ? G.st.vs : G.st.ks)[(plane + my_row(row)) / kPackedRows];
    }
    __device__ __forceinline__ void stage(uint8_t* smem, uint32_t st, uint32_t bar, int part, int64_t row, int rows16) {
      if (lane == 0) mbar_expect_tx(bar, (uint32_t)rows16 * D);
      __syncwarp();
      if (value == part) {
        uint32_t t = 0;  // of a block that is not loaded: what lies there stays finite
        const uint32_t dst = smem_u32(smem) + kOffCodes + st * kCodeBytes;
        if (rows16 == kKeys && row + kKeys <= G.a.rows) {  // the tile in one run of store rows
          constexpr int kBox = q8_box_rows(D);
          if (block == 0) {
#pragma unroll
            for (int i = 0; i < kKeys; i += kBox)
              tma_load_3d(dst + i * kPitch, part ? &G.v_box : &G.k_box, bar, 0, (int)row + i, col_head);
          }
        } else if (block * kPackedRows < rows16) {
          tma_load_3d(dst + block * (kPackedRows * kPitch), part ? &G.v : &G.k, bar, 0, (int)my_row(row), col_head);
        }
        if (block * kPackedRows < rows16) t = q8_scale_f16x2(byte);
        *reinterpret_cast<uint32_t*>(smem + kOffScales + (st * kBlocks + block) * 4) = t;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    }
  };

  // 32 dims of every 64, of two keys.  The lanes of the other half take the columns in the other order, so that
  // eight lanes meet eight 16-byte columns of the codes' swizzle as well as of the tile's.
  struct Codes {
    uint4 w[2][NH][2];  // [key0, key0 + 64][column][16 dims]
    uint32_t t[2];
  };
  struct Convert {
    const uint32_t magic;
    __device__ __forceinline__ explicit Convert(int) : magic(in_register(kQ8Magic)) {}
    __device__ __forceinline__ void read(const uint8_t* smem, uint32_t st, int, int key0, int half, Codes& x) const {
      const uint8_t* codes = smem + kOffCodes + st * kCodeBytes;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = key0 + 64 * i;
        x.t[i] = *reinterpret_cast<const uint32_t*>(smem + kOffScales + (st * kBlocks + key / kPackedRows) * 4);
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          const int c = NH == 2 ? n ^ half : n;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int chunk = 4 * c + 2 * half + j;
            const int at = D == 64 ? chunk ^ (key >> 1 & 3) : chunk ^ (key & 7);
            x.w[i][n][j] = *reinterpret_cast<const uint4*>(codes + key * kPitch + at * 16);
          }
        }
      }
    }
    __device__ __forceinline__ void write(const Codes& x, uint8_t* tile, int key0, int half) const {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 t = *reinterpret_cast<const __half2*>(&x.t[i]), z = __hmul2(t, __float2half2_rn(-1152.f));
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          const int c = NH == 2 ? n ^ half : n;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t y[4] = {x.w[i][n][j].x, x.w[i][n][j].y, x.w[i][n][j].z, x.w[i][n][j].w};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              *reinterpret_cast<uint4*>(tile + c * (128 * 128) + swz(key0 + 64 * i, half * 4 + 2 * j + k, 128)) =
                  make_uint4(q8_pair_f16<false>(y[2 * k], magic, t, z), q8_pair_f16<true>(y[2 * k], magic, t, z),
                             q8_pair_f16<false>(y[2 * k + 1], magic, t, z), q8_pair_f16<true>(y[2 * k + 1], magic, t, z));
          }
        }
      }
    }
    __device__ __forceinline__ void keys(const Codes& x, uint8_t* kt, int key0, int half) const { write(x, kt, key0, half); }
    __device__ __forceinline__ void values(const Codes& x, uint8_t* vt, int key0, int half) const { write(x, vt, key0, half); }
  };

  __device__ __forceinline__ static uint4 query(const uint4& q) {
    float amax = q8_row_amax(q, 0.f);
#pragma unroll
    for (int d = 1; d < D / 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    return q8_row_f16(q, __uint_as_float(q8_row_up(amax) << 23));
  }
  struct RowScale {
    static constexpr bool kOwn = true;
    float sl2[2];
    // the part-th of `parts` lanes that share the row (a multiple of 8 dims each); null: no such row
    __device__ __forceinline__ void set(int c, const __nv_bfloat16* q, int part, int parts, float call) {
      const int n = D / 8 / parts;
      float amax = 0.f;
      if (q) {
#pragma unroll 4
        for (int i = 0; i < n; ++i) amax = q8_row_amax(*reinterpret_cast<const uint4*>(q + (part * n + i) * 8), amax);
      }
      if (parts == 4) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      }
      sl2[c] = q8_row_scale(q8_row_up(amax), call);
    }
    __device__ __forceinline__ float get(int c, float) const { return sl2[c]; }
  };
};

template <int D>
__global__ void __launch_bounds__(kPackedTileThreads, 1) sdpa_q8_tile_kernel(const __grid_constant__ Q8AttnArgs G) {
  extern __shared__ uint8_t smem_raw[];
  packed_tile<D, Q8Tile<D>>(G, smem_raw);
}

const void* q8_tile_kernel_ptr(int D) {
  return D == 64 ? (const void*)sdpa_q8_tile_kernel<64> : (const void*)sdpa_q8_tile_kernel<128>;
}
int q8_tile_smem_bytes(int D) { return D == 64 ? Q8Tile<64>::kBytes : Q8Tile<128>::kBytes; }

}  // namespace sdpa
