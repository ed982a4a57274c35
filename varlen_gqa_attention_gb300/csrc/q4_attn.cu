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
#include <type_traits>

#include "q4.cuh"
#include "tc.cuh"

namespace sdpa {

constexpr int kQ4Consumers = 128; // threads of the four attention warps

// A unit of more than 8 rows is converted again for every 8 of them.  (16 rows a warp, twice the registers
// of output, made a CTA of 168 registers and units of 8 rows slower by a tenth; segments of more than 16
// rows have a kernel of their own, q4_tile.cu.)
template <int D>
struct Q4Cfg {
  static constexpr int kRun = D == 256 ? 2 : 4;  // 16-key blocks between two looks at the maximum
  static constexpr int kKeys = 64 * kRun;        // keys per stage of the ring
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kPerSm = D == 64 ? 3 : 2;  // CTAs per SM that registers and shared memory allow
  static constexpr int kRowBytes = D / 2;
  static constexpr int kScaleBytes = D / kQ4Group;
  static constexpr int kCodes = kKeys * kRowBytes;
  static constexpr int kScales = kKeys * kScaleBytes;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);
  static constexpr int kQPitch = D * 2 + 16;
  static constexpr int kQBytes = kSplitkRows * kQPitch;
  static constexpr int kMergeBytes = 4 * 8 * 68 * 4;  // 64 dims of the warps' rows
  static constexpr int kBytes = kStages * kStageBytes + kQBytes + kMergeBytes;
};

// One piece of a unit as the loading warp hands it on.
struct Q4Piece {
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
__device__ __forceinline__ bool q4_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
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
template <int D, typename S>
__device__ __forceinline__ void q4_unit(const AttnArgs& A, const Q4Piece& pc, int NCS, const char* ring, char* sQ,
                                        float* merge, uint32_t full, uint32_t empty, uint32_t qempty, uint32_t& it,
                                        volatile int* abort, float2* s_ml, int32_t** s_count, float* part_o,
                                        float2* part_ml) {
  constexpr int WK = D / 32;  // words of a lane's K chunk (D / 4 dims)
  constexpr int WV = D / 64;  // words of a lane's V chunk (D / 8 dims)
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
  uint4 qf[WK];
  const char* qrow = sQ + (grp * 8 + gq) * S::kQPitch + tq * (D / 2);
#pragma unroll
  for (int w = 0; w < WK; ++w) qf[w] = q4_q_order(*reinterpret_cast<const uint4*>(qrow + 16 * w));
  __syncwarp();
  if (lane == 0) mbar_arrive(qempty);

  float o[ND][4];
#pragma unroll
  for (int nd = 0; nd < ND; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, nmu[2] = {0.f, 0.f};  // nmu: added before exp2
  const float sl2 = A.scale_log2;
  const uint32_t kbits = in_register(kQ4Bf16), vbits = in_register(kQ4F16);
  // Row n of 8 keys stands for key n, with the two of every other pair swapped: the four lanes of a
  // quad then read V rows of both parities (rows of one parity share banks).
  const int kn = gq ^ ((gq >> 1) & 1);  // the key of this lane's K row
  const int ko = 2 * tq + (tq & 1);     // the keys of its V columns: ko and ko ^ 1

  for (int base = 0; base < nkeys; base += S::kKeys, ++it) {
    const uint32_t st = it % S::kStages;
    // (a wait that gave up goes on with what is there: the CTA's control flow stays whole)
    if (!mbar_try_wait(full + 8 * st, (it / S::kStages) & 1)) mbar_wait(full + 8 * st, (it / S::kStages) & 1, abort);
    const char* kc = ring + st * S::kStageBytes;
    const char* vc = kc + S::kCodes;
    const char* ks = vc + S::kCodes;
    const char* vs = ks + S::kScales;
    const int nst = min(S::kKeys, nkeys - base);
    // One run of 16 KT keys from k0 on.
    auto keys = [&](auto kt_const, int k0) {
      constexpr int KT = decltype(kt_const)::value;
      // S^T = K Q^T
      float s[KT][4];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.f;
        const int key = k0 + kt * 16 + kn;
        uint32_t kw[2][WK];  // keys key and key + 8
        __nv_bfloat162 s2[2], z2[2];
        const uint8_t* sb = reinterpret_cast<const uint8_t*>(ks) + key * S::kScaleBytes + tq * D / 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lds_words<WK>(kc + (key + 8 * h) * S::kRowBytes + tq * (D / 8), kw[h]);
          q4_scales_bf16(sb[8 * h * S::kScaleBytes], &s2[h], &z2[h]);
        }
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          if constexpr (D == 256) {
            if (w == 4) {
#pragma unroll
              for (int h = 0; h < 2; ++h) q4_scales_bf16(sb[8 * h * S::kScaleBytes + 1], &s2[h], &z2[h]);
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
            mma_bf16_16816(s[kt], a, x ? qf[w].z : qf[w].x, x ? qf[w].w : qf[w].y);
          }
        }
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
        up |= x * sl2 > m[c] + 8.f;  // false while nothing is visible
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = mx[c];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          const float mn = fmaxf(m[c], x * sl2);
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
          s[kt][e] = exp2_approx(fmaf(s[kt][e], sl2, nmu[e & 1]));
          l[e & 1] += s[kt][e];
        }

      // O^T += V^T P^T, 16 keys at a time
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const uint32_t b0 = transpose_8x8(pack_f16x2(s[kt][0], s[kt][1]));
        const uint32_t b1 = transpose_8x8(pack_f16x2(s[kt][2], s[kt][3]));
        uint32_t vw[4][WV];  // keys ko, ko ^ 1 of the first 8, then of the second
        uint32_t sb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = k0 + kt * 16 + 8 * (e >> 1) + (ko ^ (e & 1));
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
    // a stage's keys in runs; the blocks of a short last stage one by one, evenly over the warps
    if (nst > S::kKeys - 16 * S::kRun) {
#pragma unroll 1
      for (int k0 = cs * (16 * S::kRun); k0 < nst; k0 += NCS * (16 * S::kRun))
        keys(std::integral_constant<int, S::kRun>(), k0);
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
  // rows; a pass takes 8 of them.
  constexpr int kPitch = 68;  // floats: 64 dims, and a step that spreads banks
  const bool direct = ur.nslots == 1;
#pragma unroll
  for (int p = 0; p < D / 64; ++p) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float* dst = merge + (warp * 8 + 2 * tq + c) * kPitch + gq * 8;
#pragma unroll
      for (int x = 0; x < 8; x += 4) {
        const int nd = (p * 8 + x) / 2;
        *reinterpret_cast<float4*>(dst + x) = make_float4(o[nd][c], o[nd][2 + c], o[nd + 1][c], o[nd + 1][2 + c]);
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
      const int w0 = rl / 8 * NCS, rin = rl % 8;
      float M = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < NCS; ++c) M = fmaxf(M, s_ml[(w0 + c) * 8 + rin].x);
      const float Mu = M == -INFINITY ? 0.f : M;
      float L = 0.f, acc[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 1
      for (int c = 0; c < NCS; ++c) {
        const int w = (w0 + c) * 8 + rin;
        const float2 ml = s_ml[w];
        const float f = exp2_approx(ml.x - Mu);
        L += ml.y * f;
#pragma unroll
        for (int x = 0; x < 8; x += 4) {
          const float4 u = *reinterpret_cast<const float4*>(merge + w * kPitch + n * 8 + x);
          acc[x] += u.x * f; acc[x + 1] += u.y * f; acc[x + 2] += u.z * f; acc[x + 3] += u.w * f;
        }
      }
      const int d0 = n * (D / 8) + 8 * p;
      if (direct) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int64_t r = r0 + rl;
        const int64_t i = r / A.group;
        const int h = ur.hk * A.group + (int)(r % A.group);
        *reinterpret_cast<uint4*>(A.out + (ur.q_start + i) * A.o_rs + (int64_t)h * A.o_hs + d0) =
            make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                       pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
      } else {
        if (p == 0 && n == 0) part_ml[rl] = make_float2(M, L);
        float* dst = part_o + rl * D + d0;
#pragma unroll
        for (int x = 0; x < 8; x += 4)
          *reinterpret_cast<float4*>(dst + x) = make_float4(acc[x], acc[x + 1], acc[x + 2], acc[x + 3]);
      }
    }
    bar_sync_n(1, kQ4Consumers);
  }
}

// A loading warp's part of a piece: its query rows (r0 of the segment's packed rows on) and its keys through the
// ring.  The keys [pos_lo, pos_hi) begin at a multiple of 16 and span at most rows + 15 positions, so a stage
// is at most two runs of store rows, both of whole 16-row blocks.  False: a wait gave up.
template <int D, typename S>
__device__ __forceinline__ bool q4_load_piece(const Q4AttnArgs& G, const UnitRec& ur, int64_t r0, int64_t pos_lo,
                                              int64_t pos_hi, char* ring, char* sQ, uint32_t full, uint32_t empty,
                                              uint32_t qfull, uint32_t& it, volatile int* abort) {
  const AttnArgs& A = G.a;
  const int lane = threadIdx.x & 31;
  if (lane < ur.rows) {
    const int64_t r = r0 + lane;
    const int64_t i = r / A.group;
    const int h = ur.hk * A.group + (int)(r % A.group);
    bulk_load(smem_u32(sQ + lane * S::kQPitch),
              A.q + (ur.q_start + i) * A.q_rs + (int64_t)h * A.q_hs, D * 2, qfull);
  }
  const int64_t plane = ((int64_t)ur.col * A.Hkv + ur.hk) * A.rows;  // first row of the column's head
  int64_t row = pos_lo % A.rows;
  for (int64_t pos = pos_lo; pos < pos_hi; pos += S::kKeys, ++it) {
    const uint32_t st = it % S::kStages;
    if (it >= S::kStages && !q4_wait(empty + 8 * st, (it / S::kStages - 1) & 1, abort)) return false;
    const int rows16 = (int)(min((int64_t)S::kKeys, pos_hi - pos) + 15) & ~15;
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
  return true;
}

// The loading warp: walks the CTA's pieces, hands each on with its query rows, and streams its keys through the
// ring.
template <int D, typename S>
__device__ __forceinline__ void q4_load(const Q4AttnArgs& G, char* ring, char* sQ, Q4Piece* pieces, uint32_t full,
                                        uint32_t empty, uint32_t qfull, uint32_t qempty, volatile int* abort) {
  const AttnArgs& A = G.a;
  const int lane = threadIdx.x & 31;
  PieceWalk wk;
  walk_begin(wk, A.ws, kRouteSplitk, kSkQ4Few);
  UnitRec ur;
  int64_t ta, tb;
  uint32_t it = 0, sent = 0;  // stages filled, pieces whose rows were sent for
  for (uint32_t n = 0;; ++n) {
    const bool more = walk_next(wk, ur, ta, tb);
    // (the rows' buffer is free once every warp has read them; the record of the piece before that is then no
    // longer in use)
    if (n > 0 && !q4_wait(qempty, (n - 1) & 1, abort)) break;
    const int64_t pos_lo = (int64_t)ur.lo + ta * kSplitkTile;
    const int64_t pos_hi = min((int64_t)ur.lo + tb * kSplitkTile, (int64_t)ur.hi);
    const int64_t r0 = (int64_t)ur.rb * kSplitkRows;
    if (lane == 0) {
      Q4Piece& p = pieces[n & 1];
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
    if (!q4_load_piece<D, S>(G, ur, r0, pos_lo, pos_hi, ring, sQ, full, empty, qfull, it, abort)) break;
  }
  // gave up: no copy of this CTA may still be in flight when it ends
  int none = 0;
  for (uint32_t k = it > S::kStages ? it - S::kStages : 0; k < it; ++k)
    mbar_wait(full + 8 * (k % S::kStages), (k / S::kStages) & 1, &none);
  if (sent > 0) mbar_wait(qfull, (sent - 1) & 1, &none);
}

template <int D>
__global__ void __launch_bounds__(kQ4Threads, Q4Cfg<D>::kPerSm) sdpa_q4_splitk_kernel(Q4AttnArgs G) {
  using S = Q4Cfg<D>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2];
  __shared__ __align__(16) Q4Piece pieces[2];
  __shared__ float2 s_ml[4 * 8];
  __shared__ int32_t* s_count[2];
  __shared__ int s_abort;
  const AttnArgs& A = G.a;
  char* ring = smem;
  char* sQ = smem + S::kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(sQ + S::kQBytes);
  const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
  const uint32_t qfull = empty + 8 * S::kStages, qempty = qfull + 8;

  if (threadIdx.x == 0) {
    s_abort = 0;
    s_count[0] = nullptr;
    for (int k = 0; k < S::kStages; ++k) {
      mbar_init(full + 8 * k, 1);
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

  if (threadIdx.x >= kQ4Consumers) {
    q4_load<D, S>(G, ring, sQ, pieces, full, empty, qfull, qempty, &s_abort);
  } else {
    uint32_t it = 0;
    for (uint32_t n = 0;; ++n) {
      const bool got = q4_wait(qfull, n & 1, &s_abort);
      // the four warps go on together or not at all: what follows is their common control flow
      if (!bar_and(1, kQ4Consumers, got)) break;
      const Q4Piece& pc = pieces[n & 1];
      if (!pc.valid) break;
      if (threadIdx.x == 0) s_count[1] = pc.ur.nslots > 1 ? A.ws.unit_done + pc.unit : nullptr;
      // warps that share the keys of a group of rows: 4, 2 or 1
      const int groups = (pc.ur.rows + 7) / 8;
      const int64_t slot = pc.ur.slot_base + (int64_t)pc.slot * pc.ur.rows;
      q4_unit<D, S>(A, pc, groups == 1 ? 4 : groups == 2 ? 2 : 1, ring, sQ, merge, full, empty, qempty, it, &s_abort,
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
// when the ranges of a CTA are short (q4_direct in api.cu).
// What bounds it: the chain segment - rows and first keys - output (5 us in all for one token over 128 keys), then
// the conversion, as above.
template <int D>
__global__ void __launch_bounds__(kQ4Threads, Q4Cfg<D>::kPerSm) sdpa_q4_direct_kernel(Q4DirectArgs G) {
  using S = Q4Cfg<D>;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2];
  __shared__ __align__(16) Q4Piece piece;
  __shared__ float2 s_ml[4 * 8];
  __shared__ int32_t* s_count[2];
  __shared__ int4 s_seg;  // the owner's entry
  __shared__ float2 s_part[kSplitkRows];  // maxima and sums of a cluster's part
  __shared__ int s_abort, s_owner, s_dead, s_bits;
  const AttnArgs& A = G.q4.a;
  char* ring = smem;
  char* sQ = smem + S::kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(sQ + S::kQBytes);
  const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
  const uint32_t qfull = empty + 8 * S::kStages, qempty = qfull + 8;
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
    for (int k = 0; k < S::kStages; ++k) {
      mbar_init(full + 8 * k, 1);
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
  for (int i = tid; i < G.S; i += kQ4Threads) {
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
    for (int i = tid; i < G.S; i += kQ4Threads) {
      const int4 g = i == tid ? mine : entry(i, &bits);
      if (i != owner && meet(g, o)) s_dead = 1;
    }
  }
  if (blockIdx.x == 0) {  // the call's status bits
    if (__syncthreads_or(mixed)) {
      for (int i = tid; i < G.S; i += kQ4Threads) {
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
    for (int i = tid; i < A.group * (D / 8); i += kQ4Threads)
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
    if (tid >= kQ4Consumers) {
      if (!q4_load_piece<D, S>(G.q4, ur, r0, pos_lo, pos_hi, ring, sQ, full, empty, qfull, it, &s_abort)) {
        int none = 0;  // no copy of this CTA may still be in flight when it ends
        for (uint32_t k = it > S::kStages ? it - S::kStages : 0; k < it; ++k)
          mbar_wait(full + 8 * (k % S::kStages), (k / S::kStages) & 1, &none);
        mbar_wait(qfull, 0, &none);
      }
    } else {
      const bool got = q4_wait(qfull, 0, &s_abort);
      const int groups = (A.group + 7) / 8;
      // (a cluster's parts lie in the ring, whose keys have been read when the warps' runs are joined)
      if (bar_and(1, kQ4Consumers, got))
        q4_unit<D, S>(A, piece, groups == 1 ? 4 : groups == 2 ? 2 : 1, ring, sQ, merge, full, empty, qempty, it,
                      &s_abort, s_ml, s_count, reinterpret_cast<float*>(ring), s_part);
    }
  } else if (tid < A.group) {
    s_part[tid] = make_float2(-INFINITY, 0.f);
  }
  if (parts > 1) {
    cluster_sync();
    for (int i = (int)rank * kQ4Threads + tid; i < A.group * (D / 8); i += (int)parts * kQ4Threads) {
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

template __global__ void sdpa_q4_splitk_kernel<64>(Q4AttnArgs);
template __global__ void sdpa_q4_splitk_kernel<128>(Q4AttnArgs);
template __global__ void sdpa_q4_splitk_kernel<256>(Q4AttnArgs);

int q4_splitk_smem_bytes(int D) {
  switch (D) {
    case 64: return Q4Cfg<64>::kBytes;
    case 128: return Q4Cfg<128>::kBytes;
    default: return Q4Cfg<256>::kBytes;
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
