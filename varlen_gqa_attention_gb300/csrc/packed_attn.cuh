// packed_attn.cuh - attention of few rows over a column store of codes: the split-K kernel and the one without a
// schedule, for a format F (q4_attn.cu, q8_attn.cu).
//
// A format has the stages of the ring (sizes, their loading), the query rows' fragments, and the turning of 16 keys
// and 16 values into matrix operands:
//   Args            kernel arguments: AttnArgs a, choice, and what its loading takes
//   kRun kKeys kStages kPerSm kStageBytes kRingBytes kQPitch kQBytes kMerge kMergeBytes kBytes kKind
//   side(ring, st)  a stage's scales
//   kAlign          alignment of the ring in shared memory; kFull: arrivals that fill a stage
//   kOut            what the output's rows are to be multiplied by
//   Loader          start (the piece's first stage is known), stage (one stage's copies)
//   Query           a lane's fragments of its group's query row, and the scale of its score columns' rows
//   Operands        scores (S^T of 16 keys) and values (O^T of 16 keys)
#pragma once
#include <type_traits>

#include "packed.cuh"
#include "tc.cuh"

namespace sdpa {

constexpr int kPackedConsumers = 128; // threads of the four attention warps

// One piece of a unit as the loading warp hands it on.
struct PackedPiece {
  UnitRec ur;
  int64_t pos_lo, pos_hi;  // key positions; pos_lo is a multiple of 16
  int64_t r0;              // the unit's first packed row, counted from its segment's
  int64_t unit;            // index of the unit on its route
  int32_t slot, valid;     // valid 0: no more work
};

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 block of 16-bit values: a lane holds two of row lane / 4, before and after.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
// Waits for a phase unless the CTA has given up already; false when it has (or now does).  The
// lanes of a warp agree on the answer.
__device__ __forceinline__ bool piece_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, !*abort && mbar_wait(bar, parity, abort));
}

// Bytes [p, p + 4 N) of shared memory into N words.
template <int N>
__device__ __forceinline__ void lds_words(const char* p, uint32_t (&w)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// The four attention warps on one piece.  4 / NCS groups of 8 query rows; the NCS warps of a group share a
// stage's keys.  part_o, part_ml: where a piece that is one of several of its unit leaves its rows.
template <int D, typename F>
__device__ __forceinline__ void packed_unit(const AttnArgs& A, const PackedPiece& pc, int NCS, const char* ring, char* sQ,
                                        float* merge, uint32_t full, uint32_t empty, uint32_t qempty, uint32_t& it,
                                        volatile int* abort, float2* s_ml, int32_t** s_count, float* part_o,
                                        float2* part_ml) {
  constexpr int ND = D / 16;  // m16 blocks of the output

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grp = warp / NCS, cs = warp % NCS;
  const int gq = lane >> 2, tq = lane & 3;
  const UnitRec& ur = pc.ur;
  const int R = ur.rows;
  const int64_t r0 = pc.r0;
  const int64_t pos_lo = pc.pos_lo;
  const int nkeys = (int)(pc.pos_hi - pos_lo);

  // this lane's query rows, 2 tq and 2 tq + 1 of the group's 8: the keys each sees, as offsets from pos_lo:
  // [first, first + count)
  int first[2];
  uint32_t count[2];
  int lo_max = 0, hi_min = INT32_MAX;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int rl = grp * 8 + 2 * tq + c;
    first[c] = 0;
    count[c] = INT32_MAX;  // rows past the unit's: never stored, whatever they come to
    if (rl < R) {
      const RowWin w = row_window((int)((r0 + rl) / A.group), ur.q_len, ur.kv_end, ur.causal, ur.window);
      const int a = (int)min(max((int64_t)w.lo - pos_lo, (int64_t)0), (int64_t)nkeys);
      const int b = (int)min(max((int64_t)w.hi - pos_lo, (int64_t)a), (int64_t)nkeys);
      first[c] = a;
      count[c] = b - a;
      lo_max = max(lo_max, a);
      hi_min = min(hi_min, b);
    }
  }
  // keys that every row of the warp sees
  lo_max = __reduce_max_sync(0xffffffffu, lo_max);
  hi_min = __reduce_min_sync(0xffffffffu, hi_min);

  // the query row of this lane as operand fragments
  typename F::Query query(sQ + (grp * 8 + gq) * F::kQPitch, tq, A.scale_log2);
  __syncwarp();
  if (lane == 0) mbar_arrive(qempty);

  float o[ND][4];
#pragma unroll
  for (int nd = 0; nd < ND; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, nmu[2] = {0.f, 0.f};  // nmu: added before exp2
  const typename F::Operands ops(lane);
  const int kn = ops.kn;  // the key of this lane's K row

  for (int base = 0; base < nkeys; base += F::kKeys, ++it) {
    const uint32_t st = it % F::kStages;
    // (a wait that gave up goes on with what is there: the CTA's control flow stays whole)
    if (!mbar_try_wait(full + 8 * st, (it / F::kStages) & 1)) mbar_wait(full + 8 * st, (it / F::kStages) & 1, abort);
    const char* stage = ring + st * F::kStageBytes;
    const char* side = F::side(ring, st);
    const int nst = min(F::kKeys, nkeys - base);
    // One run of 16 KT keys from k0 on.
    auto keys = [&](auto kt_const, int k0) {
      constexpr int KT = decltype(kt_const)::value;
      // S^T = K Q^T
      float s[KT][4];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.f;
        ops.scores(stage, side, k0 + kt * 16, query, s[kt]);
      }

      // mask by select, online softmax in base 2 with a lazily updated maximum (O and l are only
      // rescaled when a row's maximum grows by more than 2^8)
      const int off = base + k0;
      if (off < lo_max || off + 16 * KT > hi_min) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t j = off + kt * 16 + 8 * (e >> 1) + kn - first[e & 1];
            if (j >= count[e & 1]) s[kt][e] = -INFINITY;
          }
      }
      // (the lanes compare their own scores with the maximum; only when one is beyond it are the
      // rows' maxima taken across the lanes)
      float mx[2];
      bool up = false;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = fmaxf(s[0][c], s[0][c + 2]);
#pragma unroll
        for (int kt = 1; kt < KT; ++kt) x = fmaxf(x, fmaxf(s[kt][c], s[kt][c + 2]));
        mx[c] = x;
        up |= x * query.scale(c) > m[c] + 8.f;  // false while nothing is visible
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = mx[c];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const float mn = fmaxf(m[c], x * query.scale(c));
          float alpha = 1.f;
          if (mn > m[c] + 8.f) {
            alpha = exp2_approx(m[c] - mn);
            m[c] = mn;
            nmu[c] = kF16PLift - mn;
          }
          l[c] *= alpha;
#pragma unroll
          for (int nd = 0; nd < ND; ++nd) {
            o[nd][c] *= alpha;
            o[nd][c + 2] *= alpha;
          }
        }
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[kt][e] = exp2_approx(fmaf(s[kt][e], query.scale(e & 1), nmu[e & 1]));
          l[e & 1] += s[kt][e];
        }

      // O^T += V^T P^T, 16 keys at a time
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const uint32_t b0 = transpose_8x8(pack_f16x2(s[kt][0], s[kt][1]));
        const uint32_t b1 = transpose_8x8(pack_f16x2(s[kt][2], s[kt][3]));
        ops.values(stage, side, k0 + kt * 16, b0, b1, o);
      }
    };
    // a stage's keys in runs; the blocks of a short last stage one by one, evenly over the warps
    if (nst > F::kKeys - 16 * F::kRun) {
#pragma unroll 1
      for (int k0 = cs * (16 * F::kRun); k0 < nst; k0 += NCS * (16 * F::kRun))
        keys(std::integral_constant<int, F::kRun>(), k0);
    } else {
#pragma unroll 1
      for (int k0 = cs * 16; k0 < nst; k0 += NCS * 16) keys(std::integral_constant<int, 1>(), k0);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + 8 * st);
  }

  // row sums over the lanes that share a row
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
    // a row whose scores are NaN has no maximum: it is joined as one, and comes out NaN
    if (l[c] != l[c]) m[c] = 0.f;
    if (gq == 0) s_ml[warp * 8 + 2 * tq + c] = make_float2(m[c], l[c]);
  }

  // The warps' runs are joined through shared memory.  A lane has the D / 8 dims [gq D / 8, ...) of its
  // rows; a pass takes MD of them.
  constexpr int MD = F::kMerge;
  constexpr int kPitch = 8 * MD + 4;  // floats: the dims, and a step that spreads banks
  const bool direct = ur.nslots == 1;
#pragma unroll
  for (int p = 0; p < D / (8 * MD); ++p) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float* dst = merge + (warp * 8 + 2 * tq + c) * kPitch + gq * MD;
#pragma unroll
      for (int x = 0; x < MD; x += 4) {
        const int nd = (p * MD + x) / 2;
        *reinterpret_cast<float4*>(dst + x) = make_float4(o[nd][c], o[nd][2 + c], o[nd + 1][c], o[nd + 1][2 + c]);
      }
    }
    bar_sync_n(1, kPackedConsumers);
    // the previous piece's partial slot, written a piece ago, is counted now: a release waits for
    // the CTA's earlier writes, which by now have landed
    if (p == 0 && tid == 0 && s_count[0] != nullptr) {
      red_add_release(s_count[0], 1);
      s_count[0] = nullptr;
    }
    for (int idx = tid; idx < R * 8; idx += kPackedConsumers) {
      const int rl = idx >> 3, n = idx & 7;
      const int w0 = rl / 8 * NCS, rin = rl % 8;
      float M = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < NCS; ++c) M = fmaxf(M, s_ml[(w0 + c) * 8 + rin].x);
      const float Mu = M == -INFINITY ? 0.f : M;
      float L = 0.f, acc[MD];
#pragma unroll
      for (int k = 0; k < MD; ++k) acc[k] = 0.f;
#pragma unroll 1
      for (int c = 0; c < NCS; ++c) {
        const int w = (w0 + c) * 8 + rin;
        const float2 ml = s_ml[w];
        const float f = exp2_approx(ml.x - Mu), fo = f * F::kOut;
        L += ml.y * f;
#pragma unroll
        for (int x = 0; x < MD; x += 4) {
          const float4 u = *reinterpret_cast<const float4*>(merge + w * kPitch + n * MD + x);
          acc[x] += u.x * fo; acc[x + 1] += u.y * fo; acc[x + 2] += u.z * fo; acc[x + 3] += u.w * fo;
        }
      }
      const int d0 = n * (D / 8) + MD * p;
      if (direct) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int64_t r = r0 + rl;
        const int64_t i = r / A.group;
        const int h = ur.hk * A.group + (int)(r % A.group);
        __nv_bfloat16* dst = A.out + (ur.q_start + i) * A.o_rs + (int64_t)h * A.o_hs + d0;
        if constexpr (MD >= 8) {
#pragma unroll
          for (int x = 0; x < MD; x += 8)
            *reinterpret_cast<uint4*>(dst + x) =
                make_uint4(pack_bf16x2(acc[x] * inv, acc[x + 1] * inv), pack_bf16x2(acc[x + 2] * inv, acc[x + 3] * inv),
                           pack_bf16x2(acc[x + 4] * inv, acc[x + 5] * inv),
                           pack_bf16x2(acc[x + 6] * inv, acc[x + 7] * inv));
        } else {
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
        }
      } else {
        if (p == 0 && n == 0) part_ml[rl] = make_float2(M, L);
        float* dst = part_o + rl * D + d0;
#pragma unroll
        for (int x = 0; x < MD; x += 4)
          *reinterpret_cast<float4*>(dst + x) = make_float4(acc[x], acc[x + 1], acc[x + 2], acc[x + 3]);
      }
    }
    bar_sync_n(1, kPackedConsumers);
  }
}

// A loading warp's part of a piece: its query rows (r0 of the segment's packed rows on) and its keys through the
// ring.  The keys [pos_lo, pos_hi) begin at a multiple of 16 and span at most rows + 15 positions, so a stage
// is at most two runs of store rows, both of whole 16-row blocks.  False: a wait gave up.
template <int D, typename F>
__device__ __forceinline__ bool packed_load_piece(const typename F::Args& G, const UnitRec& ur, int64_t r0, int64_t pos_lo,
                                              int64_t pos_hi, char* ring, char* sQ, uint32_t full, uint32_t empty,
                                              uint32_t qfull, uint32_t& it, volatile int* abort) {
  const AttnArgs& A = G.a;
  const int lane = threadIdx.x & 31;
  if (lane < ur.rows) {
    const int64_t r = r0 + lane;
    const int64_t i = r / A.group;
    const int h = ur.hk * A.group + (int)(r % A.group);
    bulk_load(smem_u32(sQ + lane * F::kQPitch),
              A.q + (ur.q_start + i) * A.q_rs + (int64_t)h * A.q_hs, D * 2, qfull);
  }
  int64_t row = pos_lo % A.rows;
  auto rows_at = [&](int64_t pos) { return (int)(min((int64_t)F::kKeys, pos_hi - pos) + 15) & ~15; };
  typename F::Loader loader(G, ur, lane);
  loader.start(row, rows_at(pos_lo));
  for (int64_t pos = pos_lo; pos < pos_hi; pos += F::kKeys, ++it) {
    const uint32_t st = it % F::kStages;
    if (it >= F::kStages && !piece_wait(empty + 8 * st, (it / F::kStages - 1) & 1, abort)) return false;
    const int rows16 = rows_at(pos);
    loader.stage(ring, st, full + 8 * st, row, rows16);
    row += rows16;
    if (row >= A.rows) row -= A.rows;
    if (pos + F::kKeys < pos_hi) loader.start(row, rows_at(pos + F::kKeys));
  }
  return true;
}

// The loading warp: walks the CTA's pieces, hands each on with its query rows, and streams its keys through the
// ring.
template <int D, typename F>
__device__ __forceinline__ void packed_load(const typename F::Args& G, char* ring, char* sQ, PackedPiece* pieces, uint32_t full,
                                        uint32_t empty, uint32_t qfull, uint32_t qempty, volatile int* abort) {
  const AttnArgs& A = G.a;
  const int lane = threadIdx.x & 31;
  PieceWalk wk;
  walk_begin(wk, A.ws, kRouteSplitk, F::kKind);
  UnitRec ur;
  int64_t ta, tb;
  uint32_t it = 0, sent = 0;  // stages filled, pieces whose rows were sent for
  for (uint32_t n = 0;; ++n) {
    const bool more = walk_next(wk, ur, ta, tb);
    // (the rows' buffer is free once every warp has read them; the record of the piece before that is then no
    // longer in use)
    if (n > 0 && !piece_wait(qempty, (n - 1) & 1, abort)) break;
    const int64_t pos_lo = (int64_t)ur.lo + ta * kSplitkTile;
    const int64_t pos_hi = min((int64_t)ur.lo + tb * kSplitkTile, (int64_t)ur.hi);
    const int64_t r0 = (int64_t)ur.rb * kSplitkRows;
    if (lane == 0) {
      PackedPiece& p = pieces[n & 1];
      p.valid = more;
      if (more) {
        p.ur = ur;
        p.pos_lo = pos_lo;
        p.pos_hi = pos_hi;
        p.r0 = r0;
        p.unit = wk.u - 1;  // the walk has moved past the piece's unit
        p.slot = (int32_t)(blockIdx.x - ur.g_first);
        mbar_expect_tx(qfull, (uint32_t)ur.rows * (D * 2));
      } else {
        mbar_arrive(qfull);
      }
    }
    __syncwarp();
    if (!more) return;
    sent = n + 1;
    if (!packed_load_piece<D, F>(G, ur, r0, pos_lo, pos_hi, ring, sQ, full, empty, qfull, it, abort)) break;
  }
  // gave up: no copy of this CTA may still be in flight when it ends
  int none = 0;
  for (uint32_t k = it > F::kStages ? it - F::kStages : 0; k < it; ++k)
    mbar_wait(full + 8 * (k % F::kStages), (k / F::kStages) & 1, &none);
  if (sent > 0) mbar_wait(qfull, (sent - 1) & 1, &none);
}

// The ring in a kernel's dynamic shared memory.
template <typename F>
__device__ __forceinline__ char* packed_ring(char* smem) {
  return F::kAlign > 128 ? smem + ((0u - smem_u32(smem)) & (F::kAlign - 1)) : smem;
}

template <int D, typename F>
__device__ __forceinline__ void packed_splitk(const typename F::Args& G, char* smem) {
  __shared__ __align__(8) uint64_t bars[2 * F::kStages + 2];
  __shared__ __align__(16) PackedPiece pieces[2];
  __shared__ float2 s_ml[4 * 8];
  __shared__ int32_t* s_count[2];
  __shared__ int s_abort;
  const AttnArgs& A = G.a;
  char* ring = packed_ring<F>(smem);
  char* sQ = ring + F::kRingBytes;
  float* merge = reinterpret_cast<float*>(sQ + F::kQBytes);
  const uint32_t full = smem_u32(bars), empty = full + 8 * F::kStages;
  const uint32_t qfull = empty + 8 * F::kStages, qempty = qfull + 8;

  if (threadIdx.x == 0) {
    s_abort = 0;
    s_count[0] = nullptr;
    for (int k = 0; k < F::kStages; ++k) {
      mbar_init(full + 8 * k, F::kFull);
      mbar_init(empty + 8 * k, 4);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 4);
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();  // the scheduler's output (and the prefill kernel's end)
  griddep_launch();
  if (G.choice && A.ws.hdr->sk_rows != kSplitkRows) return;

  if (threadIdx.x >= kPackedConsumers) {
    packed_load<D, F>(G, ring, sQ, pieces, full, empty, qfull, qempty, &s_abort);
  } else {
    uint32_t it = 0;
    for (uint32_t n = 0;; ++n) {
      const bool got = piece_wait(qfull, n & 1, &s_abort);
      // the four warps go on together or not at all: what follows is their common control flow
      if (!bar_and(1, kPackedConsumers, got)) break;
      const PackedPiece& pc = pieces[n & 1];
      if (!pc.valid) break;
      if (threadIdx.x == 0) s_count[1] = pc.ur.nslots > 1 ? A.ws.unit_done + pc.unit : nullptr;
      // warps that share the keys of a group of rows: 4, 2 or 1
      const int groups = (pc.ur.rows + 7) / 8;
      const int64_t slot = pc.ur.slot_base + (int64_t)pc.slot * pc.ur.rows;
      packed_unit<D, F>(A, pc, groups == 1 ? 4 : groups == 2 ? 2 : 1, ring, sQ, merge, full, empty, qempty, it, &s_abort,
                    s_ml, s_count, A.ws.part_o[kRouteSplitk] + slot * D, A.ws.part_ml[kRouteSplitk] + slot);
      // (the unit ended on a barrier of the four warps)
      if (threadIdx.x == 0) s_count[0] = s_count[1];
    }
    if (threadIdx.x == 0 && s_count[0] != nullptr) red_add_release(s_count[0], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_abort) {
    atomicOr((unsigned long long*)&A.ws.hdr->status, (unsigned long long)SDPA_DEV_TIMEOUT);
    if (A.status_dev) atomicOr(A.status_dev, SDPA_DEV_TIMEOUT);
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
  return r;
}
// All threads of a cluster; what they wrote before is visible after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}
// Shared memory of the cluster's CTA `rank`, at this CTA's address.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// A token's heads of one KV head without a schedule: a CTA, or a cluster of up to 8 that share the keys evenly,
// finds its token's segment itself and writes the output; a cluster's CTAs join their partial rows through each
// other's shared memory, a slice of the output each.  The scheduler and the joining pass even out lengths; they
// cost 8 us, and 12 on a table of more than 32 segments, which is more than the call loses by its longest range
// when the ranges of a CTA are short (packed_direct_parts in api.cu).
// What bounds it: the chain segment - rows and first keys - output (5 us in all for one token over 128 keys), then
// the conversion, as above.
template <int D, typename F>
__device__ __forceinline__ void packed_direct(const PackedDirectArgs<typename F::Args>& G, char* smem) {
  __shared__ __align__(8) uint64_t bars[2 * F::kStages + 2];
  __shared__ __align__(16) PackedPiece piece;
  __shared__ float2 s_ml[4 * 8];
  __shared__ int32_t* s_count[2];
  __shared__ int4 s_seg;  // the owner's entry
  __shared__ float2 s_part[kSplitkRows];  // maxima and sums of a cluster's part
  __shared__ int s_abort, s_owner, s_dead, s_bits;
  const AttnArgs& A = G.packed.a;
  char* ring = packed_ring<F>(smem);
  char* sQ = ring + F::kRingBytes;
  float* merge = reinterpret_cast<float*>(sQ + F::kQBytes);
  const uint32_t full = smem_u32(bars), empty = full + 8 * F::kStages;
  const uint32_t qfull = empty + 8 * F::kStages, qempty = qfull + 8;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank(), parts = cluster_size(), pair = blockIdx.x / parts;
  const int t = (int)(pair / (uint32_t)A.Hkv), hk = (int)(pair % (uint32_t)A.Hkv);

  // entry i of the table, empty unless it is valid
  auto entry = [&](int i, int32_t* bits) -> int4 {
    int4 g = __ldg(reinterpret_cast<const int4*>(G.seq_info) + i);
    const int window = G.seg_mode ? __ldg(G.seg_mode + 2 * i + 1) : A.window;
    const int32_t b = segment_bits(g.x, g.y, g.z, g.w, A.T, A.rows, A.cols, window);
    *bits |= b;
    if (b || g.y <= 0) g = make_int4(0, 0, 0, 0);
    return g;
  };
  auto meet = [](const int4& a, const int4& b) { return max(a.x, b.x) < min(a.x + a.y, b.x + b.y); };
  if (tid == 0) {
    s_abort = s_dead = s_bits = 0;
    s_owner = -1;
    s_count[0] = nullptr;
    for (int k = 0; k < F::kStages; ++k) {
      mbar_init(full + 8 * k, F::kFull);
      mbar_init(empty + 8 * k, 4);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 4);
    mbar_fence_init();
  }
  __syncthreads();
  int32_t bits = 0;
  bool mixed = false;  // the valid segments are not in row order, or share a row
  int4 mine = make_int4(0, 0, 0, 0);  // a thread keeps its first entry
  for (int i = tid; i < G.S; i += kPackedThreads) {
    const int4 g = entry(i, &bits);
    if (i == tid) mine = g;
    if (t >= g.x && t < g.x + g.y) {
      if (atomicCAS(&s_owner, -1, i) == -1) s_seg = g;
      else s_dead = 1;
    }
    if (blockIdx.x == 0 && g.y > 0) {
      int32_t other = 0;
      for (int j = i - 1; j >= 0; --j) {
        const int4 o = entry(j, &other);
        if (o.y == 0) continue;
        mixed |= o.x + o.y > g.x;
        break;
      }
    }
  }
  __syncthreads();
  const int owner = s_owner;
  if (owner >= 0) {  // a segment that shares any row with another valid one is dropped
    const int4 o = s_seg;
    for (int i = tid; i < G.S; i += kPackedThreads) {
      const int4 g = i == tid ? mine : entry(i, &bits);
      if (i != owner && meet(g, o)) s_dead = 1;
    }
  }
  if (blockIdx.x == 0) {  // the call's status bits
    if (__syncthreads_or(mixed)) {
      for (int i = tid; i < G.S; i += kPackedThreads) {
        const int4 g = i == tid ? mine : entry(i, &bits);
        for (int j = 0; j < G.S; ++j)
          if (j != i && meet(g, entry(j, &bits))) bits |= SDPA_SEG_OVERLAP;
      }
    }
    if (bits) atomicOr(&s_bits, bits);
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    A.ws.hdr->status = s_bits;
    if (A.status_dev && s_bits) atomicOr(A.status_dev, s_bits);
  }

  RowWin w{0, 0};
  UnitRec ur{};
  if (owner >= 0 && !s_dead) {
    const int4 o = s_seg;
    ur.hk = hk;
    ur.rows = A.group;
    ur.nslots = (int)parts;
    ur.q_start = o.x;
    ur.q_len = o.y;
    ur.col = o.z;
    ur.kv_end = o.w;
    ur.causal = G.seg_mode ? __ldg(G.seg_mode + 2 * owner) != 0 : A.causal;
    ur.window = G.seg_mode ? __ldg(G.seg_mode + 2 * owner + 1) : A.window;
    w = row_window(t - o.x, o.y, o.w, ur.causal, ur.window);
  }
  if (w.hi <= w.lo) {  // no segment, or no visible key
    for (int i = tid; i < A.group * (D / 8); i += kPackedThreads)
      *reinterpret_cast<uint4*>(A.out + (int64_t)t * A.o_rs + (int64_t)(hk * A.group + i / (D / 8)) * A.o_hs +
                                i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  // this CTA's keys: runs of 64, as even as they go
  const int64_t r0 = (int64_t)(t - ur.q_start) * A.group, lo = w.lo & -kPackedRows;
  const int64_t per = (udiv((int64_t)w.hi - lo + parts - 1, parts) + 63) & ~(int64_t)63;
  const int64_t pos_lo = lo + rank * per, pos_hi = min(pos_lo + per, (int64_t)w.hi);
  if (pos_lo < pos_hi) {
    if (tid == 0) {
      piece.ur = ur;
      piece.pos_lo = pos_lo;
      piece.pos_hi = pos_hi;
      piece.r0 = r0;
      mbar_expect_tx(qfull, (uint32_t)A.group * (D * 2));
    }
    __syncthreads();
    uint32_t it = 0;
    if (tid >= kPackedConsumers) {
      if (!packed_load_piece<D, F>(G.packed, ur, r0, pos_lo, pos_hi, ring, sQ, full, empty, qfull, it, &s_abort)) {
        int none = 0;  // no copy of this CTA may still be in flight when it ends
        for (uint32_t k = it > F::kStages ? it - F::kStages : 0; k < it; ++k)
          mbar_wait(full + 8 * (k % F::kStages), (k / F::kStages) & 1, &none);
        mbar_wait(qfull, 0, &none);
      }
    } else {
      const bool got = piece_wait(qfull, 0, &s_abort);
      const int groups = (A.group + 7) / 8;
      // (a cluster's parts lie in the ring, whose keys have been read when the warps' runs are joined)
      if (bar_and(1, kPackedConsumers, got))
        packed_unit<D, F>(A, piece, groups == 1 ? 4 : groups == 2 ? 2 : 1, ring, sQ, merge, full, empty, qempty, it,
                      &s_abort, s_ml, s_count, reinterpret_cast<float*>(ring), s_part);
    }
  } else if (tid < A.group) {
    s_part[tid] = make_float2(-INFINITY, 0.f);
  }
  if (parts > 1) {
    cluster_sync();
    for (int i = (int)rank * kPackedThreads + tid; i < A.group * (D / 8); i += (int)parts * kPackedThreads) {
      const int rl = i / (D / 8), d0 = i % (D / 8) * 8;
      const float* row = reinterpret_cast<const float*>(ring) + rl * D + d0;
      float M = -INFINITY, L = 0.f, acc[8];
      for (uint32_t k = 0; k < parts; ++k) M = fmaxf(M, cluster_load2(cluster_addr(&s_part[rl], k)).x);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x] = 0.f;
      for (uint32_t k = 0; k < parts; ++k) {
        const float2 ml = cluster_load2(cluster_addr(&s_part[rl], k));
        if (ml.x == -INFINITY) continue;  // a part without keys of the row has none of it
        const float f = exp2_approx(ml.x - M);
        const uint32_t at = cluster_addr(row, k);
        const float4 u = cluster_load4(at), v = cluster_load4(at + 16);
        L += ml.y * f;
        acc[0] += u.x * f; acc[1] += u.y * f; acc[2] += u.z * f; acc[3] += u.w * f;
        acc[4] += v.x * f; acc[5] += v.y * f; acc[6] += v.z * f; acc[7] += v.w * f;
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
      *reinterpret_cast<uint4*>(A.out + (int64_t)t * A.o_rs + (int64_t)(hk * A.group + rl) * A.o_hs + d0) =
          make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                     pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    }
    cluster_sync();  // a part is read by the others until here
  }
  __syncthreads();
  if (tid == 0 && s_abort) {
    atomicOr((unsigned long long*)&A.ws.hdr->status, (unsigned long long)SDPA_DEV_TIMEOUT);
    if (A.status_dev) atomicOr(A.status_dev, SDPA_DEV_TIMEOUT);
  }
}


}  // namespace sdpa
