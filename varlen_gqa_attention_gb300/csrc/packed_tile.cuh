// packed_tile.cuh - attention of several rows over a column store of codes on the tensor-memory tensor cores, for a
// format F (q4_tile.cu, where the kernel is described, and q8_tile.cu).
//
// A format has the shared memory's layout (kOff*, kBytes), the ring of codes and what turns them into operands:
//   kParts          stages of a tile: 1 (K and V together), or 2 (K, then V)
//   kFull           arrivals that fill a stage
//   kPairs          whether eight dims of an operand row lie as 0 4 1 5 2 6 3 7
//   kIdescS kOut    the product of the scores; what the output's rows are to be multiplied by
//   Loader          start (a tile's rows are known), stage (one stage's copies)
//   Codes, Convert  a lane's codes: read (a stage's), keys and values (into the tiles)
//   query           eight dims of a query row as an operand (the lanes of a row, D / 8, call it together)
//   RowScale        the scale of a row's scores: the call's, or (kOwn) set from the row
#pragma once

#include "packed.cuh"
#include "tc.cuh"

namespace sdpa {

// mbarriers
template <int STAGES>
struct PackedTileBars {
  static constexpr int K_READY = 0;   // [2] K tile written
  static constexpr int V_READY = 2;   // [2]
  static constexpr int S_FULL = 4;    // [2] S(g) done: also, K stage g % 2 may be written again
  static constexpr int P_FULL = 6;    // [2]
  static constexpr int PV_DONE = 8;   // [2] also, V stage g % 2 may be written again
  static constexpr int ML = 10;       // the halves' maxima and sums of a piece are in shared memory
  static constexpr int Q_READY = 11;
  static constexpr int Q_EMPTY = 12;  // every S of the piece is done
  static constexpr int PC_FULL = 13;  // [2] piece record written
  static constexpr int PC_EMPTY = 15; // [2] every role is past it
  static constexpr int DRAIN = 17;
  static constexpr int C_FULL = 18;                  // [stages] codes of a stage landed
  static constexpr int C_EMPTY = C_FULL + STAGES;    // [stages] the converting warps have read them
  static constexpr int N = C_EMPTY + STAGES;
};
constexpr int kTileSoftWarps = 8, kTileConvTeam = 4, kTileConvWarps = 2 * kTileConvTeam;
constexpr int kTileRoles = kTileSoftWarps + kTileConvWarps + 1;  // warps that read piece records

struct PackedTilePiece {
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

template <int D, typename F>
__device__ __forceinline__ void packed_tile(const typename F::Args& G, uint8_t* smem_raw) {
  using C = F;
  using B = PackedTileBars<F::kCodeStages>;
  __shared__ __align__(8) uint64_t s_bars[B::N];
  __shared__ __align__(16) PackedTilePiece s_piece[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_written[2];  // softmax warps whose partial rows of a piece are written
  __shared__ float2 s_ml[2][128];
  const AttnArgs& A = G.a;

  griddep_wait();  // the scheduler's output (and the prefill kernel's end)
  griddep_launch();
  if (G.choice && A.ws.hdr->sk_rows != kPackedTileRows) return;
  {
    PieceWalk probe;  // nothing to do for this CTA: leave before any set-up
    walk_begin(probe, A.ws, kRouteSplitk, F::kKind);
    if (!walk_phase(probe)) return;
  }
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem), sbar = smem_u32(s_bars);
  auto bar = [&](int i) { return sbar + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int W_CONV = kTileSoftWarps, W_LOAD = W_CONV + kTileConvWarps, W_MMA = W_LOAD + 1;
  volatile int* abort = &s_abort;
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(i), parity & 1)) return true;
    return mbar_wait(bar(i), parity & 1, abort);
  };
  // the lanes of a warp go on together or not at all
  auto all = [](bool x) { return __all_sync(0xffffffffu, x); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kCodeStages; ++s) {
      mbar_init(bar(B::C_FULL + s), F::kFull);
      mbar_init(bar(B::C_EMPTY + s), kTileConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B::K_READY + b), kTileConvTeam);
      mbar_init(bar(B::V_READY + b), kTileConvTeam);
      mbar_init(bar(B::S_FULL + b), 1);
      mbar_init(bar(B::P_FULL + b), kTileSoftWarps);
      mbar_init(bar(B::PV_DONE + b), 1);
      mbar_init(bar(B::PC_FULL + b), 1);
      mbar_init(bar(B::PC_EMPTY + b), kTileRoles);
      s_written[b] = 0;
    }
    mbar_init(bar(B::Q_READY), kTileConvWarps);
    mbar_init(bar(B::ML), kTileSoftWarps);
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
    walk_begin(wk, A.ws, kRouteSplitk, F::kKind);
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
        PackedTilePiece& p = s_piece[n & 1];
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
      int64_t row = pos_lo % A.rows;
      auto rows_at = [&](int64_t pos) { return (int)(min((int64_t)C::kKeys, pos_hi - pos) + 15) & ~15; };
      typename F::Loader loader(G, ur, lane);
      loader.start(row, rows_at(pos_lo));
      for (int64_t pos = pos_lo; ok && pos < pos_hi; pos += C::kKeys) {
        const int rows16 = rows_at(pos);
#pragma unroll
        for (int part = 0; part < F::kParts; ++part, ++it) {  // stages of a tile
          const uint32_t st = it % C::kCodeStages;
          if (it >= C::kCodeStages && !(ok = all(wait(B::C_EMPTY + st, it / C::kCodeStages - 1)))) break;
          loader.stage(smem, st, bar(B::C_FULL + st), part, row, rows16);
        }
        row += rows16;
        if (row >= A.rows) row -= A.rows;
        if (ok && pos + C::kKeys < pos_hi) loader.start(row, rows_at(pos + C::kKeys));
      }
    }
    // no copy of this CTA may be in flight when it ends (at once when all went well: the converting
    // warps have seen every stage)
    int none = 0;
    for (uint32_t k = it > (uint32_t)C::kCodeStages ? it - C::kCodeStages : 0; k < it; ++k)
      mbar_wait(bar(B::C_FULL + k % C::kCodeStages), (k / C::kCodeStages) & 1, &none);
  } else if (warp == W_MMA) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t kIdescS = F::kIdescS;
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
    const int team = (warp - W_CONV) / kTileConvTeam, cw = warp % kTileConvTeam, tid = (warp - W_CONV) * 32 + lane;
    const typename F::Convert convert(lane);
    // this lane's keys of the tile (key0 and key0 + 64), and which 32 dims of every 64 it converts: eight
    // lanes that store together then meet eight different 16-byte columns of the swizzle
    const int key0 = cw * 16 + (lane >> 1), half = lane & 1;
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      if (!(ok = all(wait(B::PC_FULL + (n & 1), n / 2)))) break;
      const PackedTilePiece& pc = s_piece[n & 1];
      const bool valid = pc.valid;
      const int tiles = valid ? (pc.nkeys + C::kKeys - 1) / C::kKeys : 0;
      const int chunks = valid ? pc.ur.rows * (D / 8) : 0;  // 16-byte chunks of the piece's query rows
      const int quarter = valid ? tile_quarter(pc.ur.rows) : 32;
      const int64_t q0 = (int64_t)pc.ur.rb * kPackedTileRows;
      const int q_start = pc.ur.q_start, hk = pc.ur.hk;
      constexpr int kQ = 4, kT = kTileConvWarps * 32;
      uint4 q[kQ];
      auto load_q = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int idx = tid + (i0 + i) * kT, rl = idx / (D / 8), c = idx % (D / 8);
          q[i] = make_uint4(0, 0, 0, 0);
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
          const uint4 y = F::query(q[i]);
          if (idx < chunks) *reinterpret_cast<uint4*>(smem + C::kOffQ + (c / 8) * (128 * 128) + swz(at, c % 8, 128)) = y;
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
        const uint32_t b = g & 1, use = g >> 1;
        uint8_t* kt = smem + C::kOffK + b * C::kTileBytes;
        uint8_t* vt = smem + C::kOffV + b * C::kTileBytes;
        typename F::Codes codes;
#pragma unroll
        for (int part = 0; part < F::kParts; ++part) {
          const uint32_t it = g * F::kParts + part, st = it % C::kCodeStages;
          if (!(ok = all(wait(B::C_FULL + st, it / C::kCodeStages)))) break;
          // (the other team's too, so that no phase goes by unseen)
          if (b == (uint32_t)team) convert.read(smem, st, part, key0, half, codes);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::C_EMPTY + st));
          if (b != (uint32_t)team) continue;
          if (part == 0) {  // K, once the scores that read this stage are done
            if (g >= 2 && !(ok = all(wait(B::S_FULL + b, use - 1)))) break;
            convert.keys(codes, kt, key0, half);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B::K_READY + b));
          }
          if (part == F::kParts - 1) {  // V, once the product that read this stage is done
            if (g >= 2 && !(ok = all(wait(B::PV_DONE + b, use - 1)))) break;
            convert.values(codes, vt, key0, half);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B::V_READY + b));
          }
        }
        if (!ok) break;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax warps
    const int hf = warp >> 2, part = warp & 3;  // half of a tile's keys; quarter of tensor memory's lanes
    const int tq = lane & 3;
    const uint32_t lane_off = (uint32_t)(part * 32) << 16;
    const uint32_t t_s = tmem + lane_off + C::kColS + hf * 64, t_o = tmem + lane_off + C::kColO;
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
      const PackedTilePiece& pc = s_piece[n & 1];
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
          const int64_t qi = udiv((int64_t)ur.rb * kPackedTileRows + row0 + 8 * c, A.group);
          const RowWin w = row_window((int)qi, ur.q_len, ur.kv_end, ur.causal, ur.window);
          first[c] = (int)min(max((int64_t)w.lo - pos_lo, (int64_t)0), (int64_t)nkeys);
          last[c] = (int)min(max((int64_t)w.hi - pos_lo, (int64_t)first[c]), (int64_t)nkeys);
        }
      }
      typename F::RowScale rs;
      if constexpr (F::RowScale::kOwn) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c > 0 && !two) continue;
          const int64_t r = (int64_t)ur.rb * kPackedTileRows + row0 + 8 * c, qi = udiv(r, A.group);
          const __nv_bfloat16* q = A.q + (ur.q_start + qi) * A.q_rs + (int64_t)(ur.hk * A.group + (int)(r - qi * A.group)) * A.q_hs;
          rs.set(c, live[c] ? q : nullptr, quads ? tq : 0, quads ? 4 : 1, A.scale_log2);
        }
      }
      auto sl2 = [&](int c) { return rs.get(c, A.scale_log2); };
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
          up |= live[c] && mx[c] * sl2(c) > m[c] + 8.f;  // false while nothing is visible
        }
        if (__any_sync(0xffffffffu, up)) {
          float alpha[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float a = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            const float mn = fmaxf(m[c], a * sl2(c));
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
              const float p0 = exp2_approx(fmaf(x[4 * k + 2 * c], sl2(c), nmu[c]));
              const float p1 = exp2_approx(fmaf(x[4 * k + 2 * c + 1], sl2(c), nmu[c]));
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
        const float mn = fmaxf(m[0], mx * sl2(0));
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
            const float p0 = exp2_approx(fmaf(x[2 * k], sl2(0), nmu[0]));
            const float p1 = exp2_approx(fmaf(x[2 * k + 1], sl2(0), nmu[0]));
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
        f[c][0] = e0 * wgt * F::kOut;
        f[c][1] = e1 * wgt * F::kOut;
        const int64_t r = (int64_t)ur.rb * kPackedTileRows + row0 + 8 * c, qi = udiv(r, A.group);
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
            const float a = o[2 * k] * f[c][0] + o1[2 * k] * f[c][1] + 0.f;
            const float b = o[2 * k + 1] * f[c][0] + o1[2 * k + 1] * f[c][1] + 0.f;
            float y0 = a, y1 = b;
            int d = 2 * tq;
            if constexpr (F::kPairs) {  // this thread has dims tq and tq + 4 of eight; with its neighbour's, two side by side
              const float y = __shfl_xor_sync(0xffffffffu, tq & 1 ? a : b, 1);
              y0 = tq & 1 ? y : a;
              y1 = tq & 1 ? b : y;
              d = tq & 1 ? tq + 3 : tq;
            }
            const int64_t at = to[c] + 32 * c32 + 8 * (k >> 1) + d;
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
            for (int k = 0; k < 16; k += 8) {
              float y[8];  // (kPairs: columns of eight dims: 0 4 1 5 2 6 3 7)
#pragma unroll
              for (int d = 0; d < 8; ++d) y[d] = o[k + (F::kPairs ? (2 * d) % 8 + d / 4 : d)];
              const int64_t at = to[0] + 32 * c32 + s + k;
              if (direct) {
                *reinterpret_cast<uint4*>(A.out + at) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                                   pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
              } else {
                *reinterpret_cast<float4*>(part_o + at) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(part_o + at + 4) = make_float4(y[4], y[5], y[6], y[7]);
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

}  // namespace sdpa
