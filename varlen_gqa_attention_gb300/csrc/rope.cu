// rope.cu - rotary positions: packed rows on their own, and a step's queries, keys and values
// rotated and written into the bf16 or the 4-bit column store.
//
// A rotated pair (a, b) becomes (a cos - b sin, a sin + b cos), cos and sin being the table's row
// of the pair's position; the gradient of that is the rotation by the opposite angle (the matrix is
// orthogonal), so the backward pass is the same kernel with sin negated.  Dims beyond the rotated
// ones pass unchanged.
//
// A result is fma(a, cos, -(b sin)) in fp32, off by at most 2^-24 of |b sin| (that product's rounding) and
// 2^-24 of itself, and is rounded to bf16 (the other one likewise: |a sin|).
// For keys that is not enough: a 4-bit code changes by a whole step at its border, so the same input
// has to fall on the same side of it whatever order a sum was taken in, and what the bf16 store
// holds is what the 4-bit one quantises.  They are the exact results rounded to fp32 and then to
// bf16: the error bound decides nearly all of them (rot_ends), the others are taken with each
// product's rounding error recovered by a fused multiply-add and the sum's by the two-sum identity
// (rot_sum).  For queries, whose neighbours are rounded to bf16 anyway, the exact way would cost
// half as many instructions again.
// A lane takes 16 dims of a head, both halves of 8 pairs: 8 angles are loaded once for all the heads
// of a row that its warp goes through, and nothing is exchanged between lanes.
//
// What bounds it: no pipe, but the latency of loads at 24 warps an SM with two passes each on their way
// (long scoreboard 4 to 6 cycles an instruction, 1.7 to 2.1 of 4 instructions a cycle, with cold caches), and
// the ramp and the uneven end of a launch of 15 to 20 us: 16384 rows of 16 x 64 take 13.1 us over buffers that are
// not in the L2 (5.2 TB/s; 10.4 us over ones that are), 4097 of 20 x 256 17.1 (5.0 TB/s; two rows for some warps, one
// for the others), 4093 tokens of 32/8 x 128 on their way into a store 21.2 (4.8 TB/s).  For a handful of rows it is
// the chain of dependent loads (segment, position, angles), which the rows' own loads start ahead of.
#include "q4.cuh"
#include "step.cuh"

namespace sdpa {

// A warp takes runs of a row's heads (`parts` runs a row), 32 / (D / 16) heads a pass, one run after
// another.  Two passes are always on their way, those of the next run when its own come to an end,
// with that run's angles and the positions of the run after it, so that the chain position - angle -
// rows is waited for once.
template <int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, 3) sdpa_rope_kernel(RopeRowsArgs A) {
  constexpr int LPH = D / 16, HPP = 32 / LPH;
  __shared__ __align__(16) float2 s_angles[kRopeThreads / 32][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hs = lane / LPH;
  const LaneDims<IL> ld(A.r.half, lane % LPH);
  const int j0 = ld.turn ? ld.j0 : 0;
  const int passes = (A.H + HPP - 1) / HPP;
  const int64_t n = A.T * A.parts, stride = (int64_t)gridDim.x * (kRopeThreads / 32);
  struct Run {
    int64_t t;
    int p0, p1;
  };
  auto run_of = [&](int64_t w) -> Run {
    if (A.parts == 1) return {w, 0, passes};
    const int64_t t = udiv(w, A.parts);
    const int part = (int)(w - t * A.parts);
    return {t, passes * part / A.parts, passes * (part + 1) / A.parts};
  };
  Row16 x[2];
  auto load = [&](Row16* y, const Run& run, int p) {
    const int h = p * HPP + hs;
    if (p < run.p1 && h < A.H) {
      const __nv_bfloat16* src = A.x + run.t * A.x_rs + (int64_t)h * A.x_hs;
      y->a = ldg16(src + ld.da);
      y->b = ldg16(src + ld.db);
    }
  };
  int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + warp;
  if (w >= n) return;
  Run run = run_of(w);
  load(&x[0], run, run.p0);
  load(&x[1], run, run.p0 + 1);
  int pos[kRopeAxes], pos1[kRopeAxes] = {0, 0, 0, 0};  // of this run's row and the next one's
  fetch_positions(A.r, run.t, 0, pos);
  if (w + stride < n) fetch_positions(A.r, run_of(w + stride).t, 0, pos1);
  bool ok = check_positions(A.r, pos);
  PairAngles pa;
  fetch_angles<D>(A.r, pos, lane, &pa);
  for (;; w += stride) {
    Angles an;
    share_angles<D>(A.r, pa, j0, lane, s_angles[warp], &an);
    if (!ok && run.p0 == 0 && lane == 0 && A.status_dev) atomicOr(A.status_dev, SDPA_ROPE_BAD_POS);
    const bool more = w + stride < n;
    const Run next = run_of(more ? w + stride : w);
    bool ok1 = true;
    if (more) {
      ok1 = check_positions(A.r, pos1);
      fetch_angles<D>(A.r, pos1, lane, &pa);
      if (w + 2 * stride < n) fetch_positions(A.r, run_of(w + 2 * stride).t, 0, pos1);
    }
    for (int p = run.p0; p < run.p1; p += 2) {
      const bool last = p + 2 >= run.p1;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int h = (p + u) * HPP + hs;
        if (p + u < run.p1 && h < A.H) {
          if (ld.turn) turn16<IL, false>(&x[u], an);
          if (!ok) x[u].a = x[u].b = make_uint4(0, 0, 0, 0);
          __nv_bfloat16* y = A.out + run.t * A.o_rs + (int64_t)h * A.o_hs;
          stg16(y + ld.da, x[u].a);
          stg16(y + ld.db, x[u].b);
        }
        if (!last)
          load(&x[u], run, p + 2 + u);
        else if (more)
          load(&x[u], next, next.p0 + u);
      }
    }
    if (!more) return;
    run = next;
    ok = ok1;
  }
}

// A lane's 8 bf16 values with NaN as 0, clamped to what the largest scale holds (7 * 1920).
__device__ __forceinline__ uint32_t q4_storable(uint32_t w) {
  __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w);
  const uint32_t clean = w & __heq2_mask(v, v);
  v = *reinterpret_cast<const __nv_bfloat162*>(&clean);
  v = __hmin2(__hmax2(v, __float2bfloat162_rn(-13440.f)), __float2bfloat162_rn(13440.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The codes of 8 values.  A code is the quotient x / s rounded to even.  The quotient comes from s's
// rounded reciprocal with one Newton step, which leaves it exact where it is a short number, as at
// a border between two codes; elsewhere it is at least 2^-11 away from one (x has 8 significant
// bits, s has 4).  Adding 1.5 * 2^23 rounds it and leaves the code's two's complement in the low bits;
// the nibble is that with its top bit turned.  |x| / s < 7.5 (see q4_scale_byte) needs no clamp.
__device__ __forceinline__ uint32_t codes8(const uint32_t (&w)[4], uint32_t scale_byte) {
  const float s = q4_scale(scale_byte), r = __frcp_rn(s);
  auto code = [&](float v) {
    float q = v * r;
    q = fmaf(fmaf(-q, s, v), r, q);
    return __float_as_uint(q + 12582912.f) & 15u;
  };
  uint32_t c = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) c |= code(bf_lo(w[k])) << (8 * k) | code(bf_hi(w[k])) << (8 * k + 4);
  return c ^ 0x88888888u;
}
// Largest magnitudes of the scale groups that a lane's two chunks belong to, from the chunks' own.
// `side`: the chunks lie side by side (dims 16 i ..), so that a group is two neighbouring lanes'; else
// they are half apart, and a group is four lanes' when half is whole groups.  Every lane calls it.
template <int LPH>
__device__ __forceinline__ void group_amax(float* ma, float* mb, bool side_by_side, int half, int lane) {
  if (side_by_side) {
    const float m = fmaxf(*ma, *mb);
    *ma = *mb = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  } else if (half % 32 == 0) {
    // (lanes past the turned ones hold side-by-side chunks, in whole groups too)
    const bool mine = 8 * (lane % LPH) < half;
    const float m = fmaxf(*ma, *mb);
    const float two = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float a = fmaxf(*ma, __shfl_xor_sync(0xffffffffu, *ma, 1));
    float b = fmaxf(*mb, __shfl_xor_sync(0xffffffffu, *mb, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 2));
    *ma = mine ? a : two;
    *mb = mine ? b : two;
  } else {
    // any other split: look each chunk of both groups up where it lies
    const int base = lane - lane % LPH, h8 = half / 8, i = lane % LPH;
    const int ca = i < h8 ? i : 2 * i, cb = i < h8 ? h8 + i : 2 * i + 1;
    float out[2] = {0.f, 0.f};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = ((g ? cb : ca) & ~3) + k;
        const int at = c < h8 ? c : c < 2 * h8 ? c - h8 : c / 2;
        const bool first = c < h8 || (c >= 2 * h8 && c % 2 == 0);
        const float va = __shfl_sync(0xffffffffu, *ma, base + at), vb = __shfl_sync(0xffffffffu, *mb, base + at);
        out[g] = fmaxf(out[g], first ? va : vb);
      }
    }
    *ma = out[0];
    *mb = out[1];
  }
}

// A step's rows: queries rotated into q_out, keys rotated and values as they are into the store.
template <int D, bool IL, bool Q4>
__global__ void __launch_bounds__(kRopeThreads, 3) sdpa_rope_append_kernel(StepArgs A) {
  constexpr int LPH = D / 16;
  __shared__ RowTable s_rows;
  __shared__ __align__(16) float2 s_angles[kRopeThreads / 32][D / 2];
  step_passes<D, IL, true>(A, blockIdx.x, s_rows, s_angles, [&](Row16& y, const LaneDims<IL>& ld, const Angles& an,
                                                                bool key, int h, int lane, int2 cell) {
    if (key && ld.turn) turn16<IL, true>(&y, an);
    if constexpr (Q4) {
      const uint32_t ca[4] = {q4_storable(y.a.x), q4_storable(y.a.y), q4_storable(y.a.z), q4_storable(y.a.w)};
      const uint32_t cb[4] = {q4_storable(y.b.x), q4_storable(y.b.y), q4_storable(y.b.z), q4_storable(y.b.w)};
      float ma = amax8(ca), mb = amax8(cb);
      group_amax<LPH>(&ma, &mb, IL, A.r.half, lane);
      const uint32_t ba = q4_scale_byte(ma), bb = q4_scale_byte(mb);
      if (h < A.Hkv) {
        const int64_t at = ((int64_t)cell.y * A.Hkv + h) * A.rows + cell.x;
        uint8_t* codes = (key ? A.q4.kc : A.q4.vc) + at * (D / 2);
        uint8_t* scales = (key ? A.q4.ks : A.q4.vs) + at * (D / kQ4Group);
        *reinterpret_cast<uint32_t*>(codes + ld.da / 2) = codes8(ca, ba);
        *reinterpret_cast<uint32_t*>(codes + ld.db / 2) = codes8(cb, bb);
        if (ld.da % kQ4Group == 0) scales[ld.da / kQ4Group] = (uint8_t)ba;
        if (ld.db % kQ4Group == 0) scales[ld.db / kQ4Group] = (uint8_t)bb;
      }
    } else if (h < A.Hkv) {
      __nv_bfloat16* z =
          (key ? A.k_store : A.v_store) + (((int64_t)cell.x * A.cols + cell.y) * A.Hkv + h) * D;
      stg16(z + ld.da, y.a);
      stg16(z + ld.db, y.b);
    }
  });
}

// The rows of a segment table read back from a 4-bit store as bf16 (exact), rows that no live
// segment holds and rows before a sequence's beginning as 0.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) sdpa_q4_unpack_kernel(StepArgs A) {
  __shared__ RowTable s_rows;
  constexpr int LPH = D / 8, U = 4;
  const int64_t t0 = (int64_t)blockIdx.x * A.cr;
  const int n = (int)min((int64_t)A.cr, A.T - t0);
  find_rows<false>(A, t0, n, &s_rows, blockIdx.x == 0);
  if (threadIdx.x < n) {
    int col = 0;
    const int64_t p = row_place(&s_rows, t0, threadIdx.x, &col);
    s_rows.cell[threadIdx.x] = p >= 0 ? make_int2((int)((uint32_t)p % (uint32_t)A.rows), col) : make_int2(-1, 0);
  }
  __syncthreads();
  const int per = A.Hkv * LPH;  // chunks of 8 dims of a row; a warp takes a row
  for (int r = threadIdx.x / 32; r < n; r += kRopeThreads / 32) {
    const int2 at = s_rows.cell[r];
    const int64_t dst = (t0 + r) * A.o_rs;
    for (int x0 = threadIdx.x % 32; x0 < per; x0 += 32 * U) {
      uint32_t kw[U], vw[U], kb[U], vb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + 32 * u, h = x / LPH, c = x % LPH;
        if (x < per && at.x >= 0) {
          const int64_t cell = ((int64_t)at.y * A.Hkv + h) * A.rows + at.x;
          kw[u] = *reinterpret_cast<const uint32_t*>(A.q4.kc + cell * (D / 2) + 4 * c);
          vw[u] = *reinterpret_cast<const uint32_t*>(A.q4.vc + cell * (D / 2) + 4 * c);
          kb[u] = A.q4.ks[cell * (D / kQ4Group) + c / 4];
          vb[u] = A.q4.vs[cell * (D / kQ4Group) + c / 4];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + 32 * u, h = x / LPH, c = x % LPH;
        if (x >= per) break;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const int64_t to = dst + (int64_t)h * A.o_hs + 8 * c;
        stg16(A.k_out + to, at.x >= 0 ? q4_words8(kw[u], kb[u]) : zero);
        stg16(A.v_out + to, at.x >= 0 ? q4_words8(vw[u], vb[u]) : zero);
      }
    }
  }
}

const void* rope_kernel_ptr(int D, bool il) {
  switch (D) {
    case 64: return il ? (const void*)sdpa_rope_kernel<64, true> : (const void*)sdpa_rope_kernel<64, false>;
    case 128: return il ? (const void*)sdpa_rope_kernel<128, true> : (const void*)sdpa_rope_kernel<128, false>;
    default: return il ? (const void*)sdpa_rope_kernel<256, true> : (const void*)sdpa_rope_kernel<256, false>;
  }
}
template <bool IL, bool Q4>
static const void* append_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_rope_append_kernel<64, IL, Q4>;
    case 128: return (const void*)sdpa_rope_append_kernel<128, IL, Q4>;
    default: return (const void*)sdpa_rope_append_kernel<256, IL, Q4>;
  }
}
const void* rope_append_kernel_ptr(int D, bool il, bool q4) {
  if (q4) return il ? append_ptr<true, true>(D) : append_ptr<false, true>(D);
  return il ? append_ptr<true, false>(D) : append_ptr<false, false>(D);
}
const void* q4_unpack_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q4_unpack_kernel<64>;
    case 128: return (const void*)sdpa_q4_unpack_kernel<128>;
    default: return (const void*)sdpa_q4_unpack_kernel<256>;
  }
}
int rope_heads_per_pass(int D) { return 32 / (D / 16); }

}  // namespace sdpa
