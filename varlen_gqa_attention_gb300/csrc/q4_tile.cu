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
// 3.5 cycles an instruction), and 576 threads leave 96 registers each, which spill (40 bytes at D = 128, 44
// at 64).  64 segments over 6144 keys on average, 8 KV heads, D = 128: 24 rows 150 us, 64
// rows 158 us.  With the rows packed (the softmax of 32 rows all in one quarter, on one scheduler) and four
// converting warps: 221 and 205 us.  (Products of 64 rows instead of 128, and codes read without bank
// conflicts, came to the same; so did rows copied to every quarter, each with its share of the keys, and one
// team converting K and the other V.  Softmax teams that take whole tiles in turn: 203 us for 64 rows: the chain
// scores - probabilities - product of a tile is then longer, and two tiles in flight do not hide it.)
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
constexpr int kQ4SoftWarps = 8, kQ4ConvTeam = 4, kQ4ConvWarps = 2 * kQ4ConvTeam;
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

// Rows of a unit in each quarter of tensor memory's 128 lanes.
__device__ __forceinline__ int tile_quarter(int rows) { return rows <= 32 ? 8 : rows <= 64 ? 16 : 32; }

// 32 consecutive keys' scores of a row: those outside [lo, hi) (offsets from the first) are masked.
__device__ __forceinline__ void tile_mask32(float (&x)[32], int lo, int hi) {
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = k >= lo && k < hi ? x[k] : -INFINITY;
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
  if (G.choice && A.ws.hdr->sk_rows != kQ4TileRows) return;
  {
    PieceWalk probe;  // nothing to do for this CTA: leave before any set-up
    walk_begin(probe, A.ws, kRouteSplitk, kSkQ4Tile);
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
      mbar_init(bar(B::K_READY + b), kQ4ConvTeam);
      mbar_init(bar(B::V_READY + b), kQ4ConvTeam);
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
    walk_begin(wk, A.ws, kRouteSplitk, kSkQ4Tile);
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
    const int team = (warp - W_CONV) / kQ4ConvTeam, cw = warp % kQ4ConvTeam, tid = (warp - W_CONV) * 32 + lane;
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
      const int quarter = valid ? tile_quarter(pc.ur.rows) : 32;
      const int64_t q0 = (int64_t)pc.ur.rb * kQ4TileRows;
      const int q_start = pc.ur.q_start, hk = pc.ur.hk;
      constexpr int kQ = 4, kT = kQ4ConvWarps * 32;
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
          const int at = rl / quarter * 32 + rl % quarter;  // its lane of tensor memory
          if (idx < chunks)
            *reinterpret_cast<uint4*>(smem + C::kOffQ + (c / 8) * (128 * 128) + swz(at, c % 8, 128)) = q4_q_order(q[i]);
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
        if (b != (uint32_t)team) {  // the other team's (seen here too, so that no phase goes by unseen)
          if (lane == 0) mbar_arrive(bar(B::C_EMPTY + st));
          continue;
        }
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
    const int hf = warp >> 2, part = warp & 3;  // half of a tile's keys; quarter of tensor memory's lanes
    const int tq = lane & 3;
    const uint32_t lane_off = (uint32_t)(part * 32) << 16;
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
      const int quarter = tile_quarter(ur.rows);
      const bool here = part * quarter < ur.rows;  // the warp has rows of this unit
      // Units of up to 64 rows: a row over the four threads of a quad, two rows (of 16 keys in a half each) a
      // thread, or one for up to 32 rows.  Larger ones: a thread a row.
      const bool quads = quarter < 32, two = quarter == 16;
      const int row0 = part * quarter + (quads ? lane >> 2 : lane);
      bool live[2];
      int first[2], last[2];  // the keys a row sees, as offsets from pos_lo
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        live[c] = row0 + 8 * c < ur.rows && (c == 0 || two);
        first[c] = last[c] = 0;
        if (live[c]) {
          const int64_t qi = udiv((int64_t)ur.rb * kQ4TileRows + row0 + 8 * c, A.group);
          const RowWin w = row_window((int)qi, ur.q_len, ur.kv_end, ur.causal, ur.window);
          first[c] = (int)min(max((int64_t)w.lo - pos_lo, (int64_t)0), (int64_t)nkeys);
          last[c] = (int)min(max((int64_t)w.hi - pos_lo, (int64_t)first[c]), (int64_t)nkeys);
        }
      }
      float m[2] = {-INFINITY, -INFINITY}, nmu[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
      // O holds the tiles up to the last one, once its product is done
      auto rescalable = [&]() -> bool {
        if (!all(wait(B::PV_DONE + ((g & 1) ^ 1), (g - 1) >> 1))) return false;
        tc_fence_after();
        return true;
      };
      auto quad_tile = [&](int j) -> bool {
        const uint32_t t = t_s + (g & 1) * 128;
        const int off = j * C::kKeys + hf * 64;
        float x[32];  // [4 k + 2 c + e]: row c, key 8 k + 2 tq + e
        tc_fence_after();
        tmem_ld_quads64(t, x);
        bool edge = false, up = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) edge |= live[c] && (first[c] > off || last[c] < off + 64);
        if (__any_sync(0xffffffffu, edge)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int lo = first[c] - off, hi = last[c] - off;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int key = 8 * (k >> 1) + 2 * tq + (k & 1);
              float& y = x[4 * (k >> 1) + 2 * c + (k & 1)];
              y = key >= lo && key < hi ? y : -INFINITY;
            }
          }
        }
        float mx[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float a = x[2 * c], b = x[2 * c + 1];
#pragma unroll
          for (int k = 1; k < 8; ++k) {
            a = fmaxf(a, x[4 * k + 2 * c]);
            b = fmaxf(b, x[4 * k + 2 * c + 1]);
          }
          mx[c] = fmaxf(a, b);
          up |= live[c] && mx[c] * sl2 > m[c] + 8.f;  // false while nothing is visible
        }
        if (__any_sync(0xffffffffu, up)) {
          float alpha[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float a = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            const float mn = fmaxf(m[c], a * sl2);
            alpha[c] = 1.f;
            if (live[c] && mn > m[c] + 8.f) {
              alpha[c] = exp2_approx(m[c] - mn);
              m[c] = mn;
              nmu[c] = kF16PLift - mn;
            }
            l[c] *= alpha[c];
          }
          if (j > 0) {
            if (!rescalable()) return false;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[16];
              tmem_ld_quads32(t_o + hf * D + 32 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= alpha[(k >> 1) & 1];
              tmem_st_quads32(t_o + hf * D + 32 * c, o);
            }
          }
        }
        uint32_t pw[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 0 || two) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float p0 = exp2_approx(fmaf(x[4 * k + 2 * c], sl2, nmu[c]));
              const float p1 = exp2_approx(fmaf(x[4 * k + 2 * c + 1], sl2, nmu[c]));
              sum[0] += p0;
              sum[1] += p1;
              pw[2 * k + c] = pack_f16x2(p0, p1);
            }
            l[c] += sum[0] + sum[1];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) pw[2 * k + c] = 0u;
          }
        }
        tmem_st_quad_pairs(t, pw);  // over the scores
        tc_fence_before();
        return true;
      };
      // a row's 64 keys in two steps of 32, read twice: once for the maximum, once for the exponentials
      auto row_tile = [&](int j) -> bool {
        const uint32_t t = t_s + (g & 1) * 128;
        const int lo = first[0] - (j * C::kKeys + hf * 64), hi = last[0] - (j * C::kKeys + hf * 64);
        const bool edge = __any_sync(0xffffffffu, live[0] && (lo > 0 || hi < 64));
        float mx = -INFINITY;
        tc_fence_after();
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          float x[32];
          tmem_ld32(t + 32 * s, x);
          if (edge) tile_mask32(x, lo - 32 * s, hi - 32 * s);
          float a = x[0], b = x[1];
#pragma unroll
          for (int k = 2; k < 32; k += 2) {
            a = fmaxf(a, x[k]);
            b = fmaxf(b, x[k + 1]);
          }
          mx = fmaxf(mx, fmaxf(a, b));
        }
        const float mn = fmaxf(m[0], mx * sl2);
        const bool up = live[0] && mn > m[0] + 8.f;  // false while nothing is visible
        if (__any_sync(0xffffffffu, up)) {
          const float alpha = up ? exp2_approx(m[0] - mn) : 1.f;
          if (up) {
            m[0] = mn;
            nmu[0] = kF16PLift - mn;
          }
          l[0] *= alpha;
          if (j > 0) {
            if (!rescalable()) return false;
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
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          float x[32];
          tmem_ld32(t + 32 * s, x);
          if (edge) tile_mask32(x, lo - 32 * s, hi - 32 * s);
          uint32_t pw[16];
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float p0 = exp2_approx(fmaf(x[2 * k], sl2, nmu[0]));
            const float p1 = exp2_approx(fmaf(x[2 * k + 1], sl2, nmu[0]));
            sum[0] += p0;
            sum[1] += p1;
            pw[k] = pack_f16x2(p0, p1);
          }
          l[0] += sum[0] + sum[1];
          tmem_st16u(t + 16 * s, pw);  // over the scores: the second 32 lie behind all of the pairs
        }
        tc_fence_before();
        return true;
      };
      for (int j = 0; j < tiles; ++j, ++g) {
        if (!(ok = all(wait(B::S_FULL + (g & 1), g >> 1)))) break;
        if (here && !(ok = quads ? quad_tile(j) : row_tile(j))) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::P_FULL + (g & 1)));
      }
      if (!ok) break;
      count_late();
      // the halves' maxima and sums change hands once the piece's last product is done: every warp has then
      // left the last piece's
      if (!(ok = all(wait(B::PV_DONE + ((g - 1) & 1), (g - 1) >> 1)))) break;
      tc_fence_after();
      const bool direct = ur.nslots == 1;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (quads) {
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 1);
          l[c] += __shfl_xor_sync(0xffffffffu, l[c], 2);
        }
        if (l[c] != l[c]) m[c] = 0.f;  // a row whose scores are NaN has no maximum: it is joined as one
        if (live[c]) s_ml[hf][row0 + 8 * c] = make_float2(m[c], l[c]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::ML));
      if (!(ok = all(wait(B::ML, n)))) break;
      if (!here) continue;
      // each half's warps write half of the dims
      float f[2][2];  // [row][half]
      int64_t to[2];  // the row's place in the output, or among the partial rows
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f[c][0] = f[c][1] = 0.f;
        to[c] = 0;
        if (!live[c]) continue;
        const float2 ml0 = s_ml[0][row0 + 8 * c], ml1 = s_ml[1][row0 + 8 * c];
        const float M = fmaxf(ml0.x, ml1.x), Mu = M == -INFINITY ? 0.f : M;
        const float e0 = exp2_approx(ml0.x - Mu), e1 = exp2_approx(ml1.x - Mu);
        const float L = ml0.y * e0 + ml1.y * e1;
        // (a row that sees no key has zeros of either sign in O: its products were of P = 0)
        const float wgt = !direct ? 1.f : L == 0.f ? 0.f : 1.f / L;
        f[c][0] = e0 * wgt;
        f[c][1] = e1 * wgt;
        const int64_t r = (int64_t)ur.rb * kQ4TileRows + row0 + 8 * c, qi = udiv(r, A.group);
        const int64_t pidx = ur.slot_base + (int64_t)slot * ur.rows + row0 + 8 * c;
        if (direct) {
          const int h = ur.hk * A.group + (int)(r - qi * A.group);
          to[c] = (ur.q_start + qi) * A.o_rs + (int64_t)h * A.o_hs + hf * (D / 2);
        } else {
          to[c] = pidx * D + hf * (D / 2);
          if (hf == 0 && (!quads || tq == 0)) A.ws.part_ml[kRouteSplitk][pidx] = make_float2(M, L);
        }
      }
      float* part_o = A.ws.part_o[kRouteSplitk];
#pragma unroll 1
      for (int c32 = 0; c32 < D / 64; ++c32) {
        if (quads) {
          float o[16], o1[16];
          tmem_ld_quads32(t_o + hf * (D / 2) + 32 * c32, o);
          tmem_ld_quads32(t_o + D + hf * (D / 2) + 32 * c32, o1);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = k & 1;
            // this thread has dims tq and tq + 4 of eight; with its neighbour's, two side by side
            const float a = o[2 * k] * f[c][0] + o1[2 * k] * f[c][1] + 0.f;
            const float b = o[2 * k + 1] * f[c][0] + o1[2 * k + 1] * f[c][1] + 0.f;
            const float y = __shfl_xor_sync(0xffffffffu, tq & 1 ? a : b, 1);
            const float y0 = tq & 1 ? y : a, y1 = tq & 1 ? b : y;
            const int64_t at = to[c] + 32 * c32 + 8 * (k >> 1) + (tq & 1 ? tq + 3 : tq);
            if (!live[c]) continue;
            if (direct)
              *reinterpret_cast<uint32_t*>(A.out + at) = pack_bf16x2(y0, y1);
            else
              *reinterpret_cast<float2*>(part_o + at) = make_float2(y0, y1);
          }
        } else {
#pragma unroll 1
          for (int s = 0; s < 32; s += 16) {
            float o[16], o1[16];
            __syncwarp();
            tmem_ld16(t_o + hf * (D / 2) + 32 * c32 + s, o);
            tmem_ld16(t_o + D + hf * (D / 2) + 32 * c32 + s, o1);
            if (!live[0]) continue;
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = o[k] * f[0][0] + o1[k] * f[0][1] + 0.f;
#pragma unroll
            for (int k = 0; k < 16; k += 8) {  // columns of eight dims: 0 4 1 5 2 6 3 7
              const float* y = o + k;
              const int64_t at = to[0] + 32 * c32 + s + k;
              if (direct) {
                *reinterpret_cast<uint4*>(A.out + at) = make_uint4(pack_bf16x2(y[0], y[2]), pack_bf16x2(y[4], y[6]),
                                                                   pack_bf16x2(y[1], y[3]), pack_bf16x2(y[5], y[7]));
              } else {
                *reinterpret_cast<float4*>(part_o + at) = make_float4(y[0], y[2], y[4], y[6]);
                *reinterpret_cast<float4*>(part_o + at + 4) = make_float4(y[1], y[3], y[5], y[7]);
              }
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      if (!direct) {
        late = A.ws.unit_done + unit;
        late_warps = 2 * ((ur.rows + quarter - 1) / quarter);
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
