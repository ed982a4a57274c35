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
//     128 keys) into a ring of stages, across the borders of pieces, so that the next piece's
//     first keys (and its query rows) travel while this one is finished;
//   * no value is written back to shared memory: codes are read once per warp, as whole words, in
//     an order that makes them operand fragments at once.  The contraction over dims does not care
//     about their order, so a lane of K takes D / 4 dims of its key side by side (with their one
//     or two scales), and the query fragments follow; a lane of V takes D / 8 dims side by side of
//     four keys, and the output's columns follow;
//   * scales are multiplied in by the conversion's own fused multiply-add, exactly.
// P is rounded to fp16 (half a step is at most 2^-11 of it, against 2^-8 in bf16) and V is exact in
// fp16; Q and K are multiplied in bf16, where both are exact.  Sums are fp32.  The lazily updated
// maximum leaves P at most 2^8 above it, so P is kept 2^7 times larger, its sum too: at most 2^15,
// and a row's largest at least 2^7, so that a P that fp16's smallest step (2^-24) cannot hold is
// less than 2^-32 of its row: a million such keys are still lost in the output's rounding.
#include "q4.cuh"
#include "tc.cuh"

namespace sdpa {

constexpr int kQ4Stage = 128;     // keys per stage of the ring
constexpr int kQ4Consumers = 128; // threads of the four attention warps
constexpr float kQ4PLift = 7.f;    // P is held 2^7 times larger
constexpr int kQ4MergePitch = 68; // floats per row of the merge buffer: 64 and a step that spreads banks

template <int D>
struct Q4Smem {
  static constexpr int kRowBytes = D / 2;
  static constexpr int kScaleBytes = D / kQ4Group;
  static constexpr int kStages = 4;
  static constexpr int kQBufs = 2;
  // CTAs per SM that registers (the output alone is D / 2 of them) and shared memory allow
  static constexpr int kPerSm = D == 64 ? 3 : D == 128 ? 2 : 1;
  static constexpr int kCodes = kQ4Stage * kRowBytes;
  static constexpr int kScales = kQ4Stage * kScaleBytes;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);
  static constexpr int kQPitch = D * 2 + 16;
  static constexpr int kQBytes = kSplitkRows * kQPitch;
  static constexpr int kMergeBytes = 4 * 16 * kQ4MergePitch * 4;
  static constexpr int kBytes = kStages * kStageBytes + kQBufs * kQBytes + kMergeBytes;
};

// One piece of a unit as the loading warp hands it on.
struct Q4Piece {
  UnitRec ur;
  int64_t pos_lo, pos_hi;  // key positions; pos_lo is a multiple of 16
  int64_t unit;            // index of the unit on its route
  int32_t slot, valid;     // valid 0: no more work
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// D(16x8 f32) += A(16x16 f16, row) * B(16x8 f16, col)
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Waits for a phase unless the CTA has given up already; false when it has (or now does).  The
// lanes of a warp agree on the answer.
__device__ __forceinline__ bool q4_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, !*abort && mbar_wait(bar, parity, abort));
}

// The query rows' operand fragments for one word (8 dims) of a lane's K chunk: two k-steps.
// The conversion pairs nibbles i and i + 4, so the fragments pair dims i and i + 4.
__device__ __forceinline__ void q4_q_frags(const char* row0, const char* row8, uint32_t (&f)[2][4]) {
  const uint4 a = *reinterpret_cast<const uint4*>(row0);
  const uint4 b = *reinterpret_cast<const uint4*>(row8);
  f[0][0] = __byte_perm(a.x, a.z, 0x5410);
  f[0][2] = __byte_perm(a.x, a.z, 0x7632);
  f[1][0] = __byte_perm(a.y, a.w, 0x5410);
  f[1][2] = __byte_perm(a.y, a.w, 0x7632);
  f[0][1] = __byte_perm(b.x, b.z, 0x5410);
  f[0][3] = __byte_perm(b.x, b.z, 0x7632);
  f[1][1] = __byte_perm(b.y, b.w, 0x5410);
  f[1][3] = __byte_perm(b.y, b.w, 0x7632);
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

// The four attention warps on one piece: 16 packed rows (mt) x every NCS-th run of 32 keys (cs).
template <int D, int NCS>
__device__ __forceinline__ void q4_unit(const AttnArgs& A, const Q4Piece& pc, const char* ring, const char* sQ,
                                        float* merge, uint32_t full, uint32_t empty, uint32_t& it,
                                        volatile int* abort, float2* s_ml, int32_t** s_count) {
  using S = Q4Smem<D>;
  constexpr int WK = D / 32;  // words of a lane's K chunk (D / 4 dims)
  constexpr int WV = D / 64;  // words of a lane's V chunk (D / 8 dims)
  constexpr int ND = D / 8;   // n8 blocks of the output
  constexpr bool kQRegs = D <= 128;  // query fragments stay in registers

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mt = warp / NCS, cs = warp % NCS;
  const int gq = lane >> 2, tq = lane & 3;
  const UnitRec& ur = pc.ur;
  const int R = ur.rows;
  const int64_t r0 = (int64_t)ur.rb * kSplitkRows;
  const int64_t pos_lo = pc.pos_lo, pos_hi = pc.pos_hi;

  // this lane's two rows: local rows mt*16 + gq and +8
  int32_t rlo[2], rhi[2];
  bool live[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int rl = mt * 16 + gq + 8 * e;
    live[e] = rl < R;
    rlo[e] = INT32_MIN;  // rows past the unit's: never stored, whatever they come to
    rhi[e] = INT32_MAX;
    if (live[e]) {
      const RowWin w = row_window((int)((r0 + rl) / A.group), ur.q_len, ur.kv_end, ur.causal, ur.window);
      rlo[e] = (int32_t)max((int64_t)w.lo, pos_lo);
      rhi[e] = (int32_t)min((int64_t)w.hi, pos_hi);
    }
  }
  const int32_t lo_max = max(rlo[0], rlo[1]), hi_min = min(rhi[0], rhi[1]);

  const char* q0 = sQ + (mt * 16 + gq) * S::kQPitch + tq * (D / 2);
  uint32_t qf[kQRegs ? WK : 1][2][4];
  if constexpr (kQRegs) {
#pragma unroll
    for (int w = 0; w < WK; ++w) q4_q_frags(q0 + 16 * w, q0 + 8 * S::kQPitch + 16 * w, qf[w]);
  }

  float o[ND][4];
#pragma unroll
  for (int nd = 0; nd < ND; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float sl2 = A.scale_log2;
  // Column n of an 8-key block stands for key n, with the two of every other pair swapped: the
  // four lanes of a quad then read V rows of both parities (rows of one parity share banks).
  const int kn = gq ^ ((gq >> 1) & 1);        // the key of this lane's K column
  const int ko = 2 * tq + (tq & 1);           // the keys of its two score columns: ko and ko ^ 1

  for (int64_t base = pos_lo; base < pos_hi; base += kQ4Stage, ++it) {
    const uint32_t st = it % S::kStages;
    q4_wait(full + 8 * st, (it / S::kStages) & 1, abort);
    const char* kc = ring + st * S::kStageBytes;
    const char* vc = kc + S::kCodes;
    const char* ks = vc + S::kCodes;
    const char* vs = ks + S::kScales;
    const int nst = (int)min((int64_t)kQ4Stage, pos_hi - base);
#pragma unroll 1
    for (int k0 = cs * 32; k0 < nst; k0 += NCS * 32) {
      // S = Q K^T over 32 keys
      float s[4][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const int key = k0 + nb * 8 + kn;
        uint32_t kw[WK];
        lds_words<WK>(kc + key * S::kRowBytes + tq * (D / 8), kw);
        __nv_bfloat162 s2, z2;
        const uint8_t* sb = reinterpret_cast<const uint8_t*>(ks) + key * S::kScaleBytes + tq * D / 128;
        q4_scales_bf16(sb[0], &s2, &z2);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          if constexpr (D == 256) {
            if (w == 4) q4_scales_bf16(sb[1], &s2, &z2);
          }
          uint32_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = q4_pair_bf16(kw[w] >> (4 * i), s2, z2);
          if constexpr (kQRegs) {
            mma_bf16_16816(s[nb], qf[w][0], b[0], b[1]);
            mma_bf16_16816(s[nb], qf[w][1], b[2], b[3]);
          } else {
            uint32_t f[2][4];
            q4_q_frags(q0 + 16 * w, q0 + 8 * S::kQPitch + 16 * w, f);
            mma_bf16_16816(s[nb], f[0], b[0], b[1]);
            mma_bf16_16816(s[nb], f[1], b[2], b[3]);
          }
        }
      }

      // mask by select, online softmax in base 2 with a lazily updated maximum (O and l are only
      // rescaled when a row's maximum grows by more than 2^8)
      const int64_t tile0 = base + k0;
      const bool all = tile0 >= lo_max && tile0 + 32 <= hi_min;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = e >> 1;
          float x = s[nb][e];
          if (!all) {
            const int64_t j = tile0 + nb * 8 + (ko ^ (e & 1));
            x = !live[rr] || (j >= rlo[rr] && j < rhi[rr]) ? x : -INFINITY;
          }
          s[nb][e] = x;
          mx[rr] = fmaxf(mx[rr], x);
        }
      }
      float alpha[2], nmu[2];
      bool resc = false;
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 1));
        mx[rr] = fmaxf(mx[rr], __shfl_xor_sync(0xffffffffu, mx[rr], 2));
        const float mn = fmaxf(m[rr], mx[rr] * sl2);
        const bool up = mn > m[rr] + 8.f;  // false while nothing is visible
        alpha[rr] = up ? exp2_approx(m[rr] - mn) : 1.f;
        if (up) m[rr] = mn;
        resc |= up;
        nmu[rr] = m[rr] == -INFINITY ? 0.f : kQ4PLift - m[rr];
      }
      float ls[2] = {0.f, 0.f};
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = exp2_approx(fmaf(s[nb][e], sl2, nmu[e >> 1]));
          s[nb][e] = p;
          ls[e >> 1] += p;
        }
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) l[rr] = l[rr] * alpha[rr] + ls[rr];
      if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
        for (int nd = 0; nd < ND; ++nd) {
          o[nd][0] *= alpha[0];
          o[nd][1] *= alpha[0];
          o[nd][2] *= alpha[1];
          o[nd][3] *= alpha[1];
        }
      }

      // O += P V, 16 keys at a time
#pragma unroll
      for (int bp = 0; bp < 2; ++bp) {
        uint32_t a[4];
        a[0] = pack_f16x2(s[2 * bp][0], s[2 * bp][1]);
        a[1] = pack_f16x2(s[2 * bp][2], s[2 * bp][3]);
        a[2] = pack_f16x2(s[2 * bp + 1][0], s[2 * bp + 1][1]);
        a[3] = pack_f16x2(s[2 * bp + 1][2], s[2 * bp + 1][3]);
        const int key = k0 + bp * 16;
        uint32_t vw[4][WV];  // keys ko, ko ^ 1 of the first block, then of the second
        uint32_t sb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = key + 8 * (e >> 1) + (ko ^ (e & 1));
          lds_words<WV>(vc + k * S::kRowBytes + gq * (D / 16), vw[e]);
          sb[e] = reinterpret_cast<const uint8_t*>(vs)[k * S::kScaleBytes + gq * D / 256];
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
            for (int i = 0; i < 4; ++i) {
              const uint32_t y0 = i < 2 ? x0 << (6 - 4 * i) : x0 >> (4 * i - 6);
              const uint32_t y1 = i < 2 ? x1 << (6 - 4 * i) : x1 >> (4 * i - 6);
              mma_f16_16816(o[8 * w + 4 * hf + i], a, q4_pair_f16(y0, s2[0], z2[0]),
                            q4_pair_f16(y1, s2[1], z2[1]));
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + 8 * st);
  }

  // row sums over the quad
#pragma unroll
  for (int rr = 0; rr < 2; ++rr) {
    l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 1);
    l[rr] += __shfl_xor_sync(0xffffffffu, l[rr], 2);
    // a row whose scores are NaN has no maximum: it is joined as one, and comes out NaN
    if (l[rr] != l[rr]) m[rr] = 0.f;
  }
  if (tq == 0) {
    s_ml[warp * 16 + gq] = make_float2(m[0], l[0]);
    s_ml[warp * 16 + gq + 8] = make_float2(m[1], l[1]);
  }

  // The warps' runs are joined through shared memory, 64 dims at a time: output block nd of column
  // n is dim n * (D / 8) + nd, so a pass over 8 blocks is 8 dims side by side of every column.
  const bool direct = ur.nslots == 1;
#pragma unroll
  for (int p = 0; p < D / 64; ++p) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* dst = merge + (warp * 16 + gq + 8 * e) * kQ4MergePitch + (2 * tq + c) * 8;
        const int x = 2 * e + c;
        *reinterpret_cast<float4*>(dst) =
            make_float4(o[8 * p][x], o[8 * p + 1][x], o[8 * p + 2][x], o[8 * p + 3][x]);
        *reinterpret_cast<float4*>(dst + 4) =
            make_float4(o[8 * p + 4][x], o[8 * p + 5][x], o[8 * p + 6][x], o[8 * p + 7][x]);
      }
    }
    bar_sync_n(1, kQ4Consumers);
    // the previous piece's partial slot, written a piece ago, is counted now: a release waits for
    // the CTA's earlier writes, which by now have landed
    if (p == 0 && tid == 0 && s_count[0] != nullptr) {
      red_add_release(s_count[0], 1);
      s_count[0] = nullptr;
    }
    for (int idx = tid; idx < R * 8; idx += kQ4Consumers) {
      const int rl = idx >> 3, n = idx & 7;
      const int mtr = rl / 16, rin = rl % 16;
      float M = -INFINITY;
#pragma unroll
      for (int c = 0; c < NCS; ++c) M = fmaxf(M, s_ml[(mtr * NCS + c) * 16 + rin].x);
      const float Mu = M == -INFINITY ? 0.f : M;
      float L = 0.f, acc[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll
      for (int c = 0; c < NCS; ++c) {
        const int w = (mtr * NCS + c) * 16 + rin;
        const float2 ml = s_ml[w];
        const float f = exp2_approx(ml.x - Mu);
        L += ml.y * f;
        const float* src = merge + w * kQ4MergePitch + n * 8;
        const float4 u0 = *reinterpret_cast<const float4*>(src);
        const float4 u1 = *reinterpret_cast<const float4*>(src + 4);
        acc[0] += u0.x * f; acc[1] += u0.y * f; acc[2] += u0.z * f; acc[3] += u0.w * f;
        acc[4] += u1.x * f; acc[5] += u1.y * f; acc[6] += u1.z * f; acc[7] += u1.w * f;
      }
      const int d0 = n * (D / 8) + 8 * p;
      if (direct) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int64_t r = r0 + rl;
        const int64_t i = r / A.group;
        const int h = ur.hk * A.group + (int)(r % A.group);
        uint4 pk;
        pk.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        pk.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
        pk.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
        pk.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4*>(A.out + (ur.q_start + i) * A.o_rs + (int64_t)h * A.o_hs + d0) = pk;
      } else {
        const int64_t pi = ur.slot_base + (int64_t)pc.slot * R + rl;
        if (p == 0 && n == 0) A.ws.part_ml[kRouteSplitk][pi] = make_float2(M, L);
        float* dst = A.ws.part_o[kRouteSplitk] + pi * D + d0;
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
      }
    }
    bar_sync_n(1, kQ4Consumers);
  }
}

// The loading warp: walks the CTA's pieces, hands each on with its query rows, and streams its keys
// through the ring.  A piece's keys [pos_lo, pos_hi) begin at a multiple of 16 and span at most
// rows + 15 positions, so a stage is at most two runs of store rows, both of whole 16-row blocks.
template <int D>
__device__ __forceinline__ void q4_load(const Q4AttnArgs& G, char* ring, char* sQ, Q4Piece* pieces, uint32_t full,
                                        uint32_t empty, uint32_t qfull, uint32_t qempty, volatile int* abort) {
  using S = Q4Smem<D>;
  const AttnArgs& A = G.a;
  const int lane = threadIdx.x & 31;
  PieceWalk wk;
  walk_begin(wk, A.ws, kRouteSplitk);
  UnitRec ur;
  int64_t ta, tb;
  uint32_t it = 0, n = 0;
  for (;; ++n) {
    const bool more = walk_next(wk, ur, ta, tb);
    const uint32_t b = n % S::kQBufs;
    if (n >= S::kQBufs && !q4_wait(qempty + 8 * b, (n / S::kQBufs - 1) & 1, abort)) break;
    const int64_t pos_lo = (int64_t)ur.lo + ta * kSplitkTile;
    const int64_t pos_hi = min((int64_t)ur.lo + tb * kSplitkTile, (int64_t)ur.hi);
    if (lane == 0) {
      Q4Piece& p = pieces[b];
      p.valid = more;
      if (more) {
        p.ur = ur;
        p.pos_lo = pos_lo;
        p.pos_hi = pos_hi;
        p.unit = wk.u - 1;  // the walk has moved past the piece's unit
        p.slot = (int32_t)(blockIdx.x - ur.g_first);
        mbar_expect_tx(qfull + 8 * b, (uint32_t)ur.rows * (D * 2));
      } else {
        mbar_arrive(qfull + 8 * b);
      }
    }
    __syncwarp();
    if (!more) return;
    if (lane < ur.rows) {
      const int64_t r = (int64_t)ur.rb * kSplitkRows + lane;
      const int64_t i = r / A.group;
      const int h = ur.hk * A.group + (int)(r % A.group);
      bulk_load(smem_u32(sQ + b * S::kQBytes + lane * S::kQPitch),
                A.q + (ur.q_start + i) * A.q_rs + (int64_t)h * A.q_hs, D * 2, qfull + 8 * b);
    }
    const int64_t plane = ((int64_t)ur.col * A.Hkv + ur.hk) * A.rows;  // first row of the column's head
    int64_t row = pos_lo % A.rows;
    bool ok = true;
    for (int64_t pos = pos_lo; pos < pos_hi; pos += kQ4Stage, ++it) {
      const uint32_t st = it % S::kStages;
      if (it >= S::kStages && !(ok = q4_wait(empty + 8 * st, (it / S::kStages - 1) & 1, abort))) break;
      const int rows16 = (int)(min((int64_t)kQ4Stage, pos_hi - pos) + 15) & ~15;
      const int first = (int)min((int64_t)rows16, A.rows - row), second = rows16 - first;
      if (lane == 0) {
        const uint32_t bar = full + 8 * st;
        const uint32_t dst = smem_u32(ring + st * S::kStageBytes);
        mbar_expect_tx(bar, (uint32_t)rows16 * 2 * (S::kRowBytes + S::kScaleBytes));
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint8_t* codes = v ? G.st.vc : G.st.kc;
          const uint8_t* scales = v ? G.st.vs : G.st.ks;
          const uint32_t dc = dst + v * S::kCodes, ds = dst + 2 * S::kCodes + v * S::kScales;
          bulk_load(dc, codes + (plane + row) * S::kRowBytes, first * S::kRowBytes, bar);
          bulk_load(ds, scales + (plane + row) * S::kScaleBytes, first * S::kScaleBytes, bar);
          if (second > 0) {
            bulk_load(dc + first * S::kRowBytes, codes + plane * S::kRowBytes, second * S::kRowBytes, bar);
            bulk_load(ds + first * S::kScaleBytes, scales + plane * S::kScaleBytes, second * S::kScaleBytes, bar);
          }
        }
      }
      row += rows16;
      if (row >= A.rows) row -= A.rows;
    }
    if (!ok) break;
  }
  // gave up: no copy of this CTA may still be in flight when it ends
  int none = 0;
  for (uint32_t k = it > S::kStages ? it - S::kStages : 0; k < it; ++k)
    mbar_wait(full + 8 * (k % S::kStages), (k / S::kStages) & 1, &none);
  for (uint32_t k = n > S::kQBufs ? n - S::kQBufs : 0; k < n; ++k)
    mbar_wait(qfull + 8 * (k % S::kQBufs), (k / S::kQBufs) & 1, &none);
}

template <int D>
__global__ void __launch_bounds__(kQ4Threads, Q4Smem<D>::kPerSm) sdpa_q4_splitk_kernel(Q4AttnArgs G) {
  using S = Q4Smem<D>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2 * S::kQBufs];
  __shared__ __align__(16) Q4Piece pieces[S::kQBufs];
  __shared__ float2 s_ml[4 * 16];
  __shared__ int32_t* s_count[2];
  __shared__ int s_abort;
  const AttnArgs& A = G.a;
  char* ring = smem;
  char* sQ = smem + S::kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(sQ + S::kQBufs * S::kQBytes);
  const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
  const uint32_t qfull = empty + 8 * S::kStages, qempty = qfull + 8 * S::kQBufs;

  if (threadIdx.x == 0) {
    s_abort = 0;
    s_count[0] = nullptr;
    for (int k = 0; k < S::kStages; ++k) {
      mbar_init(full + 8 * k, 1);
      mbar_init(empty + 8 * k, 4);
    }
    for (int k = 0; k < S::kQBufs; ++k) {
      mbar_init(qfull + 8 * k, 1);
      mbar_init(qempty + 8 * k, 4);
    }
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();  // the scheduler's output (and the prefill kernel's end)
  griddep_launch();

  if (threadIdx.x >= kQ4Consumers) {
    q4_load<D>(G, ring, sQ, pieces, full, empty, qfull, qempty, &s_abort);
  } else {
    uint32_t it = 0;
    for (uint32_t n = 0;; ++n) {
      const uint32_t b = n % S::kQBufs;
      const bool got = q4_wait(qfull + 8 * b, (n / S::kQBufs) & 1, &s_abort);
      // the four warps go on together or not at all: what follows is their common control flow
      if (!bar_and(1, kQ4Consumers, got)) break;
      const Q4Piece& pc = pieces[b];
      if (!pc.valid) break;
      if (threadIdx.x == 0) s_count[1] = pc.ur.nslots > 1 ? A.ws.unit_done + pc.unit : nullptr;
      if (pc.ur.rows <= 16)
        q4_unit<D, 4>(A, pc, ring, sQ + b * S::kQBytes, merge, full, empty, it, &s_abort, s_ml, s_count);
      else
        q4_unit<D, 2>(A, pc, ring, sQ + b * S::kQBytes, merge, full, empty, it, &s_abort, s_ml, s_count);
      // (the unit ended on a barrier of the four warps)
      if (threadIdx.x == 0) s_count[0] = s_count[1];
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(qempty + 8 * b);
    }
    if (threadIdx.x == 0 && s_count[0] != nullptr) red_add_release(s_count[0], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_abort) {
    atomicOr((unsigned long long*)&A.ws.hdr->status, (unsigned long long)SDPA_DEV_TIMEOUT);
    if (A.status_dev) atomicOr(A.status_dev, SDPA_DEV_TIMEOUT);
  }
}

template __global__ void sdpa_q4_splitk_kernel<64>(Q4AttnArgs);
template __global__ void sdpa_q4_splitk_kernel<128>(Q4AttnArgs);
template __global__ void sdpa_q4_splitk_kernel<256>(Q4AttnArgs);

int q4_splitk_smem_bytes(int D) {
  switch (D) {
    case 64: return Q4Smem<64>::kBytes;
    case 128: return Q4Smem<128>::kBytes;
    default: return Q4Smem<256>::kBytes;
  }
}

const void* q4_splitk_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q4_splitk_kernel<64>;
    case 128: return (const void*)sdpa_q4_splitk_kernel<128>;
    default: return (const void*)sdpa_q4_splitk_kernel<256>;
  }
}

}  // namespace sdpa
