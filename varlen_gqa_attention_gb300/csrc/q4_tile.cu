// q4_tile.cu - attention over the 4-bit column store for segments of several rows (draft blocks, short
// chunks), on the tensor-memory tensor cores; D = 64 and 128.
//
// The split-K kernel of q4_attn.cu turns every key into operands once for 8 query rows; a block of 16
// draft rows with 4 heads a KV head is 64, and converting is what that kernel does most.  Here a key is
// converted once for up to 128 rows: S = Q K^T (128 rows x 128 keys) and O += P V are tcgen05 products, Q,
// K and V in shared memory, S, P and O in tensor memory.  Per CTA (one per SM), 14 warps:
//   * a loading warp walks the CTA's pieces (the split-K route's, in units of 128 packed rows and tiles of
//     128 keys), hands them on, and streams their codes and scales into a ring by bulk copies;
//   * four converting warps turn a tile's codes into bf16 K and fp16 V tiles (exactly: see q4.cuh),
//     written in the 128-byte swizzle that the products read, and a piece's query rows likewise;
//   * one warp issues the products: S(0) S(1) | PV(0) S(2) | PV(1) S(3) ...  P lies over the scores it came
//     from, which the next scores of that buffer overwrite behind PV (one thread's products run in order);
//   * eight softmax warps, a thread a row (= tensor-memory lane), four for a tile's first 64 keys and four
//     for the others.  The two halves keep a maximum, a sum and an output of their own, as if they were two
//     CTAs' pieces, and are joined when the piece ends: nothing passes between them in between.  A warp
//     none of whose rows exist skips its work, so that a unit of 64 rows costs half of one of 128.
// A word of codes gives its values in pairs (dim i, dim i + 4); K and V tiles keep that order, and so do
// the query rows, and the output's columns are put in order as they are written.
// P is fp16, held 2^7 times larger, as in q4_attn.cu.
//
// Bound by the issue slots and by each role's own latency: a tile at D = 128 is about 1.8 thousand warp
// instructions of conversion and 0.9 thousand for each 32 rows of softmax.  With one warp a row quarter
// for all 128 keys (half the softmax warps, twice the converting ones) a tile of 64 rows took 3.7 thousand
// cycles, waiting for its two softmax warps: 16 segments of 64 rows over 3100 keys 55 us, and 45 us so.  (K a
// tile ahead of V, and the converting warps off the partitions that the softmax of few rows has to run on,
// came to the same.)
#include "q4.cuh"
#include "tc.cuh"

namespace sdpa {

template <int D>
struct Q4TileCfg {
  static constexpr int kRowBytes = D / 2;
  static constexpr int kScaleBytes = D / kQ4Group;
  static constexpr int kKeys = kQ4TileKeys;
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
};

// mbarriers
struct Q4TileBars {
  static constexpr int C_FULL = 0;    // [3] codes of a stage landed
  static constexpr int C_EMPTY = 3;   // [3] the converting warps have read them
  static constexpr int K_READY = 6;   // [2] K tile written
  static constexpr int V_READY = 8;   // [2]
  static constexpr int S_FULL = 10;   // [2] S(g) done: also, K stage g % 2 may be written again
  static constexpr int P_FULL = 12;   // [2]
  static constexpr int PV_DONE = 14;  // [2] also, V stage g % 2 may be written again
  static constexpr int ML = 16;       // the halves' maxima and sums of a piece are in shared memory
  static constexpr int Q_READY = 18;
  static constexpr int Q_EMPTY = 19;  // every S of the piece is done
  static constexpr int PC_FULL = 20;  // [2] piece record written
  static constexpr int PC_EMPTY = 22; // [2] every role is past it
  static constexpr int DRAIN = 24;
  static constexpr int N = 25;
};
constexpr int kQ4SoftWarps = 8, kQ4ConvWarps = 4;
constexpr int kQ4TileRoles = kQ4SoftWarps + kQ4ConvWarps + 1;  // warps that read piece records

struct Q4TilePiece {
  UnitRec ur;
  int64_t pos_lo;   // a multiple of 16
  int64_t unit;
  int32_t nkeys, slot, valid, pad;
};

// fp16 A and B, fp32 accumulation, B MN-major
constexpr uint32_t kIdescPV64 = (1u << 4) | (1u << 16) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPV128 = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// 64 consecutive keys' scores of a row: those outside [lo, hi) (offsets from the first) are masked.
__device__ __forceinline__ void tile_mask64(float (&x)[64], int lo, int hi) {
#pragma unroll
  for (int k = 0; k < 64; ++k) x[k] = k >= lo && k < hi ? x[k] : -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(kQ4TileThreads, 1) sdpa_q4_tile_kernel(Q4AttnArgs G) {
  using C = Q4TileCfg<D>;
  using B = Q4TileBars;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[B::N];
  __shared__ __align__(16) Q4TilePiece s_piece[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_written[2];  // softmax warps whose partial rows of a piece are written
  __shared__ float2 s_ml[2][128];
  const AttnArgs& A = G.a;

  griddep_wait();  // the scheduler's output (and the prefill kernel's end)
  griddep_launch();
  {
    PieceWalk probe;  // nothing to do for this CTA: leave before any set-up
    walk_begin(probe, A.ws, kRouteSplitk);
    if (!walk_phase(probe)) return;
  }
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem), sbar = smem_u32(s_bars);
  auto bar = [&](int i) { return sbar + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int W_CONV = kQ4SoftWarps, W_LOAD = W_CONV + kQ4ConvWarps, W_MMA = W_LOAD + 1;
  volatile int* abort = &s_abort;
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity & 1)) return true;
    return mbar_wait(bar(i), parity & 1, abort);
  };
  // the lanes of a warp go on together or not at all
  auto all = [](bool x) { return __all_sync(0xffffffffu, x); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(bar(B::C_FULL + s), 1);
      mbar_init(bar(B::C_EMPTY + s), kQ4ConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B::K_READY + b), kQ4ConvWarps);
      mbar_init(bar(B::V_READY + b), kQ4ConvWarps);
      mbar_init(bar(B::S_FULL + b), 1);
      mbar_init(bar(B::P_FULL + b), kQ4SoftWarps);
      mbar_init(bar(B::PV_DONE + b), 1);
      mbar_init(bar(B::PC_FULL + b), 1);
      mbar_init(bar(B::PC_EMPTY + b), kQ4TileRoles);
      s_written[b] = 0;
    }
    mbar_init(bar(B::Q_READY), kQ4ConvWarps);
    mbar_init(bar(B::ML), kQ4SoftWarps);
    mbar_init(bar(B::Q_EMPTY), 1);
    mbar_init(bar(B::DRAIN), 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  if (warp == W_LOAD) {
    // ---------------------------------------------------------------- loading warp
    PieceWalk wk;
    walk_begin(wk, A.ws, kRouteSplitk);
    UnitRec ur;
    int64_t ta, tb;
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const bool more = walk_next(wk, ur, ta, tb);
      if (n >= 2 && !(ok = all(wait(B::PC_EMPTY + (n & 1), n / 2 - 1)))) break;
      const int64_t pos_lo = (int64_t)ur.lo + ta * C::kKeys;
      const int64_t pos_hi = min((int64_t)ur.lo + tb * C::kKeys, (int64_t)ur.hi);
      if (lane == 0) {
        Q4TilePiece& p = s_piece[n & 1];
        p.valid = more;
        if (more) {
          p.ur = ur;
          p.pos_lo = pos_lo;
          p.nkeys = (int32_t)(pos_hi - pos_lo);
          p.unit = wk.u - 1;  // the walk has moved past the piece's unit
          p.slot = (int32_t)(blockIdx.x - ur.g_first);
        }
        mbar_arrive(bar(B::PC_FULL + (n & 1)));
      }
      __syncwarp();
      if (!more) break;
      // a tile is at most two runs of store rows, both of whole 16-row blocks (pos_lo is a multiple of 16,
      // a unit spans at most rows + 15 positions)
      const int64_t plane = ((int64_t)ur.col * A.Hkv + ur.hk) * A.rows;
      int64_t row = pos_lo % A.rows;
      for (int64_t pos = pos_lo; pos < pos_hi; pos += C::kKeys, ++it) {
        const uint32_t st = it % C::kCodeStages;
        if (it >= C::kCodeStages &&
            !(ok = all(wait(B::C_EMPTY + st, it / C::kCodeStages - 1))))
          break;
        const int rows16 = (int)(min((int64_t)C::kKeys, pos_hi - pos) + 15) & ~15;
        const int first = (int)min((int64_t)rows16, A.rows - row), second = rows16 - first;
        if (lane == 0) {
          const uint32_t dst = sbase + C::kOffCodes + st * C::kCodeBytes;
          mbar_expect_tx(bar(B::C_FULL + st), (uint32_t)rows16 * 2 * (C::kRowBytes + C::kScaleBytes));
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint8_t* codes = v ? G.st.vc : G.st.kc;
            const uint8_t* scales = v ? G.st.vs : G.st.ks;
            const uint32_t dc = dst + v * C::kCodes, ds = dst + 2 * C::kCodes + v * C::kScales;
            bulk_load(dc, codes + (plane + row) * C::kRowBytes, first * C::kRowBytes, bar(B::C_FULL + st));
            bulk_load(ds, scales + (plane + row) * C::kScaleBytes, first * C::kScaleBytes, bar(B::C_FULL + st));
            if (second > 0) {
              bulk_load(dc + first * C::kRowBytes, codes + plane * C::kRowBytes, second * C::kRowBytes,
                        bar(B::C_FULL + st));
              bulk_load(ds + first * C::kScaleBytes, scales + plane * C::kScaleBytes, second * C::kScaleBytes,
                        bar(B::C_FULL + st));
            }
          }
        }
        row += rows16;
        if (row >= A.rows) row -= A.rows;
      }
    }
    // no copy of this CTA may be in flight when it ends (at once when all went well: the converting
    // warps have seen every stage)
    int none = 0;
    for (uint32_t k = it > (uint32_t)C::kCodeStages ? it - C::kCodeStages : 0; k < it; ++k)
      mbar_wait(bar(B::C_FULL + k % C::kCodeStages), (k / C::kCodeStages) & 1, &none);
  } else if (warp == W_MMA) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t kIdescPV = D == 64 ? kIdescPV64 : kIdescPV128;
    const uint64_t q_desc = sdesc_sw128(sbase + C::kOffQ, 16, 1024);
    const uint64_t k_desc = sdesc_sw128(sbase + C::kOffK, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sbase + C::kOffV, 128 * 128, 1024);
    auto issue_s = [&](uint32_t g) -> bool {
      const uint32_t b = g & 1, use = g >> 1;
      if (!all(wait(B::K_READY + b, use))) return false;
      tc_fence_after();
      const uint64_t kd = k_desc + (uint64_t)((b * C::kTileBytes) >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
        tc_mma_ss_w(tmem + C::kColS + b * 128, q_desc + off, kd + off, kIdescS, k > 0 ? 1u : 0u);
      }
      tc_commit_w(bar(B::S_FULL + b));
      return true;
    };
    uint32_t g0 = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      if (!(ok = all(wait(B::PC_FULL + (n & 1), n / 2)))) break;
      const bool valid = s_piece[n & 1].valid;
      const int tiles = valid ? (s_piece[n & 1].nkeys + C::kKeys - 1) / C::kKeys : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::PC_EMPTY + (n & 1)));
      if (!valid) break;
      if (!(ok = all(wait(B::Q_READY, n)))) break;
      ok = issue_s(g0) && (tiles < 2 || issue_s(g0 + 1));
      if (ok && tiles <= 2) tc_commit_w(bar(B::Q_EMPTY));
      for (int j = 0; ok && j < tiles; ++j) {
        const uint32_t g = g0 + j, b = g & 1, use = g >> 1;
        if (!(ok = all(wait(B::P_FULL + b, use) && wait(B::V_READY + b, use)))) break;
        tc_fence_after();
        const uint64_t vd = v_desc + (uint64_t)((b * C::kTileBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc_mma_ts_w(tmem + C::kColO + (k >> 2) * D, tmem + C::kColS + b * 128 + (k >> 2) * 64 + 8 * (k & 3),
                      vd + (uint64_t)((k * 16 * 128) >> 4), kIdescPV, j > 0 || (k & 3) ? 1u : 0u);
        tc_commit_w(bar(B::PV_DONE + b));
        if (j + 2 < tiles) {
          if (!(ok = issue_s(g + 2))) break;
          if (j + 3 == tiles) tc_commit_w(bar(B::Q_EMPTY));
        }
      }
      g0 += tiles;
    }
    // wait (bounded) until every product issued here is done
    tc_commit_w(bar(B::DRAIN));
    int none = 0;
    mbar_wait(bar(B::DRAIN), 0, &none);
    __syncwarp();
  } else if (warp >= W_CONV) {
    // ---------------------------------------------------------------- converting warps
    const int cw = warp - W_CONV, tid = cw * 32 + lane;
    const uint32_t kbits = in_register(kQ4Bf16), vbits = in_register(kQ4F16);
    // this lane's keys of the tile (key0 and key0 + 64), and which 32 dims of every 64 it converts: eight
    // lanes that store together then meet eight different 16-byte columns of the swizzle
    const int key0 = cw * 16 + (lane >> 1), half = lane & 1;
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      if (!(ok = all(wait(B::PC_FULL + (n & 1), n / 2)))) break;
      const Q4TilePiece& pc = s_piece[n & 1];
      const bool valid = pc.valid;
      const int tiles = valid ? (pc.nkeys + C::kKeys - 1) / C::kKeys : 0;
      const int chunks = valid ? pc.ur.rows * (D / 8) : 0;  // 16-byte chunks of the piece's query rows
      const int64_t q0 = (int64_t)pc.ur.rb * kQ4TileRows;
      const int q_start = pc.ur.q_start, hk = pc.ur.hk;
      constexpr int kQ = 8, kT = kQ4ConvWarps * 32;
      uint4 q[kQ];
      auto load_q = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int idx = tid + (i0 + i) * kT, rl = idx / (D / 8), c = idx % (D / 8);
          if (idx < chunks) {
            const int64_t r = q0 + rl, t = udiv(r, A.group);
            const int h = hk * A.group + (int)(r - t * A.group);
            q[i] = *reinterpret_cast<const uint4*>(A.q + (q_start + t) * A.q_rs + (int64_t)h * A.q_hs + 8 * c);
          }
        }
      };
      auto store_q = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int idx = tid + (i0 + i) * kT, rl = idx / (D / 8), c = idx % (D / 8);
          if (idx < chunks)
            *reinterpret_cast<uint4*>(smem + C::kOffQ + (c / 8) * (128 * 128) + swz(rl, c % 8, 128)) = q4_q_order(q[i]);
        }
      };
      load_q(0);  // in flight until the last piece's scores are done
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::PC_EMPTY + (n & 1)));
      if (!valid) break;
      if (n > 0 && !(ok = all(wait(B::Q_EMPTY, n - 1)))) break;
      store_q(0);
      for (int i0 = kQ; i0 * kT < chunks; i0 += kQ) {
        load_q(i0);
        store_q(i0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::Q_READY));

      for (int j = 0; j < tiles; ++j, ++g) {
        const uint32_t st = g % C::kCodeStages, b = g & 1, use = g >> 1;
        if (!(ok = all(wait(B::C_FULL + st, g / C::kCodeStages)))) break;
        const uint8_t* codes = smem + C::kOffCodes + st * C::kCodeBytes;
        const uint8_t* scales = codes + 2 * C::kCodes;
        constexpr int NH = D / 64;  // 64-dim columns of the tile
        uint4 w[2][2][NH];          // [K, V][key0, key0 + 64]
        uint32_t sb[2][2][NH];
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int c = 0; c < NH; ++c) {
              const int key = key0 + 64 * x;
              w[v][x][c] =
                  *reinterpret_cast<const uint4*>(codes + v * C::kCodes + key * C::kRowBytes + c * 32 + half * 16);
              sb[v][x][c] = scales[v * C::kScales + key * C::kScaleBytes + c * 2 + half];
            }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::C_EMPTY + st));
        // K, once the scores that read this stage are done
        if (g >= 2 && !(ok = all(wait(B::S_FULL + b, use - 1)))) break;
        uint8_t* kt = smem + C::kOffK + b * C::kTileBytes;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int c = 0; c < NH; ++c) {
            __nv_bfloat162 s2, z2;
            q4_scales_bf16(sb[0][x][c], &s2, &z2);
            const uint32_t y[4] = {w[0][x][c].x, w[0][x][c].y, w[0][x][c].z, w[0][x][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(kt + c * (128 * 128) + swz(key0 + 64 * x, half * 4 + i, 128)) =
                  make_uint4(q4_pair_bf16(y[i], kbits, s2, z2), q4_pair_bf16(y[i] >> 4, kbits, s2, z2),
                             q4_pair_bf16(y[i] >> 8, kbits, s2, z2), q4_pair_bf16(y[i] >> 12, kbits, s2, z2));
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::K_READY + b));
        // V, once the product that read this stage is done
        if (g >= 2 && !(ok = all(wait(B::PV_DONE + b, use - 1)))) break;
        uint8_t* vt = smem + C::kOffV + b * C::kTileBytes;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int c = 0; c < NH; ++c) {
            __half2 s2, z2;
            q4_scales_f16(sb[1][x][c], sb[1][x][c], &s2, &z2);
            const uint32_t y[4] = {w[1][x][c].x, w[1][x][c].y, w[1][x][c].z, w[1][x][c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(vt + c * (128 * 128) + swz(key0 + 64 * x, half * 4 + i, 128)) =
                  make_uint4(q4_pair_f16(y[i] << 6, vbits, s2, z2), q4_pair_f16(y[i] << 2, vbits, s2, z2),
                             q4_pair_f16(y[i] >> 2, vbits, s2, z2), q4_pair_f16(y[i] >> 6, vbits, s2, z2));
          }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::V_READY + b));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax warps
    const int hf = warp >> 2, row = (warp & 3) * 32 + lane;  // half of the tile's keys; row of the unit
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + C::kColS + hf * 64, t_o = tmem + lane_off + C::kColO;
    const float sl2 = A.scale_log2;
    // a piece's partial rows, written a piece ago, are counted in the next one's epilogue: by then the
    // fence has nothing to wait for.  The last of the warps that wrote some counts the slot.
    int32_t* late = nullptr;
    int late_warps = 0, late_at = 0;
    auto count_late = [&]() {
      if (late == nullptr) return;
      __threadfence();
      __syncwarp();
      if (lane == 0 && atomicAdd(&s_written[late_at], 1) == late_warps - 1) {
        s_written[late_at] = 0;
        __threadfence();
        red_add_release(late, 1);
      }
      late = nullptr;
    };
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      if (!(ok = all(wait(B::PC_FULL + (n & 1), n / 2)))) break;
      const Q4TilePiece& pc = s_piece[n & 1];
      if (!pc.valid) break;
      const UnitRec ur = pc.ur;
      const int nkeys = pc.nkeys, slot = pc.slot;
      const int64_t pos_lo = pc.pos_lo, unit = pc.unit;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::PC_EMPTY + (n & 1)));
      const int tiles = (nkeys + C::kKeys - 1) / C::kKeys;
      const bool here = (warp & 3) * 32 < ur.rows;  // the warp has rows of this unit
      const bool live = row < ur.rows;
      const int64_t r = (int64_t)ur.rb * kQ4TileRows + row;
      const int64_t qi = udiv(r, A.group);
      int first = 0, last = 0;  // the keys the row sees, as offsets from pos_lo
      if (live) {
        const RowWin w = row_window((int)qi, ur.q_len, ur.kv_end, ur.causal, ur.window);
        first = (int)min(max((int64_t)w.lo - pos_lo, (int64_t)0), (int64_t)nkeys);
        last = (int)min(max((int64_t)w.hi - pos_lo, (int64_t)first), (int64_t)nkeys);
      }
      float m = -INFINITY, nmu = 0.f, l = 0.f;
      for (int j = 0; j < tiles; ++j, ++g) {
        const uint32_t b = g & 1, use = g >> 1;
        if (!(ok = all(wait(B::S_FULL + b, use)))) break;
        if (here) {
          const int off = j * C::kKeys + hf * 64, lo = first - off, hi = last - off;
          tc_fence_after();
          float x[64];
          tmem_ld64(t_s + b * 128, x);
          if (__any_sync(0xffffffffu, live && (lo > 0 || hi < 64))) tile_mask64(x, lo, hi);
          float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int k = 4; k < 64; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], x[k]);
          const float mn = fmaxf(m, fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2);
          const bool up = live && mn > m + 8.f;  // false while nothing is visible
          if (__any_sync(0xffffffffu, up)) {
            const float alpha = up ? exp2_approx(m - mn) : 1.f;
            if (up) {
              m = mn;
              nmu = kQ4PLift - mn;
            }
            l *= alpha;
            if (j > 0) {  // O holds the tiles up to the last one, once its product is done
              if (!(ok = all(wait(B::PV_DONE + (b ^ 1), (g - 1) >> 1)))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(t_o + hf * D + 32 * c, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= alpha;
                tmem_st32(t_o + hf * D + 32 * c, o);
              }
            }
          }
          uint32_t pw[32];
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float p0 = exp2_approx(fmaf(x[2 * k], sl2, nmu)), p1 = exp2_approx(fmaf(x[2 * k + 1], sl2, nmu));
            sum[(2 * k) & 3] += p0;
            sum[(2 * k + 1) & 3] += p1;
            pw[k] = pack_f16x2(p0, p1);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st32u(t_s + b * 128, pw);  // over the scores
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::P_FULL + b));
      }
      if (!ok) break;
      count_late();
      // the halves' maxima and sums change hands once the piece's last product is done: every warp has then
      // left the last piece's
      if (!(ok = all(wait(B::PV_DONE + ((g - 1) & 1), (g - 1) >> 1)))) break;
      tc_fence_after();
      if (l != l) m = 0.f;  // a row whose scores are NaN has no maximum: it is joined as one
      s_ml[hf][row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::ML));
      if (!(ok = all(wait(B::ML, n)))) break;
      if (!here) continue;
      const float2 ml0 = s_ml[0][row], ml1 = s_ml[1][row];
      const float M = fmaxf(ml0.x, ml1.x), Mu = M == -INFINITY ? 0.f : M;
      const float e0 = exp2_approx(ml0.x - Mu), e1 = exp2_approx(ml1.x - Mu);
      const float L = ml0.y * e0 + ml1.y * e1;
      const bool direct = ur.nslots == 1;
      const bool empty = L == 0.f;  // a row that sees no key writes zeros (never 0 * O)
      const float wgt = direct ? 1.f / L : 1.f;
      const float f0 = e0 * wgt, f1 = e1 * wgt;
      const int h = ur.hk * A.group + (int)(r - qi * A.group);
      // each half's warps write half of the dims
      __nv_bfloat16* orow = A.out + (ur.q_start + qi) * A.o_rs + (int64_t)h * A.o_hs + hf * (D / 2);
      const int64_t pidx = ur.slot_base + (int64_t)slot * ur.rows + row;
      float* prow = A.ws.part_o[kRouteSplitk] + pidx * D + hf * (D / 2);
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        float o[32], o1[32];
        __syncwarp();
        tmem_ld32(t_o + hf * (D / 2) + 32 * c, o);
        tmem_ld32(t_o + D + hf * (D / 2) + 32 * c, o1);
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = empty ? 0.f : o[k] * f0 + o1[k] * f1;
#pragma unroll
        for (int k = 0; k < 32; k += 8) {  // columns of eight dims: 0 4 1 5 2 6 3 7
          const float* y = o + k;
          if (direct) {
            *reinterpret_cast<uint4*>(orow + 32 * c + k) =
                make_uint4(pack_bf16x2(y[0], y[2]), pack_bf16x2(y[4], y[6]), pack_bf16x2(y[1], y[3]),
                           pack_bf16x2(y[5], y[7]));
          } else {
            *reinterpret_cast<float4*>(prow + 32 * c + k) = make_float4(y[0], y[2], y[4], y[6]);
            *reinterpret_cast<float4*>(prow + 32 * c + k + 4) = make_float4(y[1], y[3], y[5], y[7]);
          }
        }
      }
      tc_fence_before();
      if (!direct) {
        if (live && hf == 0) A.ws.part_ml[kRouteSplitk][pidx] = make_float2(M, L);
        late = A.ws.unit_done + unit;
        late_warps = 2 * ((ur.rows + 31) / 32);
        late_at = n & 1;
      }
    }
    if (ok) count_late();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && s_abort) {
    atomicOr((unsigned long long*)&A.ws.hdr->status, (unsigned long long)SDPA_DEV_TIMEOUT);
    if (A.status_dev) atomicOr(A.status_dev, SDPA_DEV_TIMEOUT);
  }
  if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

template __global__ void sdpa_q4_tile_kernel<64>(Q4AttnArgs);
template __global__ void sdpa_q4_tile_kernel<128>(Q4AttnArgs);

const void* q4_tile_kernel_ptr(int D) {
  return D == 64 ? (const void*)sdpa_q4_tile_kernel<64> : (const void*)sdpa_q4_tile_kernel<128>;
}
int q4_tile_smem_bytes(int D) { return D == 64 ? Q4TileCfg<64>::kBytes : Q4TileCfg<128>::kBytes; }

}  // namespace sdpa
