// rope.cu - rotary positions: packed rows on their own, and a step's queries, keys and values
// rotated and written into the bf16 or the 4-bit column store.
//
// A rotated pair (a, b) becomes (a cos - b sin, a sin + b cos), cos and sin being the table's row
// of the pair's position; the gradient of that is the rotation by the opposite angle (the matrix is
// orthogonal), so the backward pass is the same kernel with sin negated.  Dims beyond the rotated
// ones pass unchanged.
//
// Products of a bf16 value and an fp32 cosine have 32 significant bits, and their difference can
// cancel: each product's rounding error is recovered by a fused multiply-add and each sum's by the
// two-sum identity, so that a result is the exact one rounded to fp32 (and then to bf16).  A 4-bit
// code changes by a whole step at its border, so the same input has to fall on the same side of it
// whatever order a sum was taken in.
//
// What bounds it: the rows' bytes, read once and written once (a lane holds 8 dims of a head, its
// pairs' other halves come from a neighbour lane by shuffle, never by a second load), and for a
// handful of rows the chain of dependent loads (segment, position, angles, row).
#include "q4.cuh"
#include "rope.cuh"

namespace sdpa {

// fp32 value of a * c + b * s, rounded once (up to 2^-47 of the larger product).
__device__ __forceinline__ float rot_sum(float a, float c, float b, float s) {
  const float p = a * c, q = b * s;
  const float e = fmaf(a, c, -p), f = fmaf(b, s, -q);
  const float d = p + q;
  const float t = d - p;
  const float g = (p - (d - t)) + (q - t);
  const float r = d + (g + (e + f));
  return fabsf(d) < INFINITY ? r : d;  // an infinite row stays what it is: its error terms are NaN
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// What a lane needs to turn dims [8c, 8c + 8) of any head of one row.
struct LaneTurn {
  float cs[8], sn[8];  // half-split pairs: one per dim; interleaved: the first four, one per pair
  int partner;         // lane with the pairs' other halves (half-split)
  bool turn, second;   // the dims are rotated at all; they are the pairs' second halves
};

// Angles of chunk c of a row whose positions are pos[axis].  LPH: lanes per head.
template <bool IL>
__device__ __forceinline__ void lane_turn(const RopeArgs& R, const int (&pos)[kRopeAxes], int c, int lane,
                                          LaneTurn* t) {
  constexpr int N = IL ? 4 : 8;
  const int d0 = 8 * c, half = R.half;
  t->turn = d0 < 2 * half;
  t->second = !IL && d0 >= half;
  t->partner = lane;
  if (!t->turn) return;
  const int hc = half / 8;
  if (!IL) t->partner = t->second ? lane - hc : lane + hc;
  const int j0 = IL ? d0 / 2 : (t->second ? d0 - half : d0);
  auto axis_pos = [&](int j) {
    int p = pos[0];
#pragma unroll
    for (int a = 1; a < kRopeAxes; ++a) p = j >= R.sec_end[a - 1] ? pos[a] : p;
    return p;
  };
  const int pf = axis_pos(j0), pl = axis_pos(j0 + N - 1);
  if (pf == pl) {
    const float4* src = reinterpret_cast<const float4*>(R.table + (int64_t)pf * half + j0);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      const float4 v = __ldg(src + k);
      t->cs[2 * k] = v.x; t->sn[2 * k] = v.y;
      t->cs[2 * k + 1] = v.z; t->sn[2 * k + 1] = v.w;
    }
    if constexpr (N > 2) {
      // a section that begins and ends inside the chunk has a position of its own between them
      bool mixed = false;
#pragma unroll
      for (int k = 1; k < N - 1; ++k) mixed |= axis_pos(j0 + k) != pf;
      if (!mixed) {
        if (R.inverse) {
#pragma unroll
          for (int k = 0; k < N; ++k) t->sn[k] = -t->sn[k];
        }
        return;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float2 v = __ldg(R.table + (int64_t)axis_pos(j0 + k) * half + j0 + k);
    t->cs[k] = v.x;
    t->sn[k] = R.inverse ? -v.y : v.y;
  }
}

// Turns a lane's 8 dims.  Every lane of the warp calls it (shuffles).
template <bool IL>
__device__ __forceinline__ uint4 turn8(const uint4& x, const LaneTurn& t) {
  const uint32_t own[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
  if constexpr (IL) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = bf_lo(own[k]), b = bf_hi(own[k]);
      r[k] = pack_bf16x2(rot_sum(a, t.cs[k], b, -t.sn[k]), rot_sum(b, t.cs[k], a, t.sn[k]));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t o = __shfl_sync(0xffffffffu, own[k], t.partner);
      const float s0 = t.second ? t.sn[2 * k] : -t.sn[2 * k], s1 = t.second ? t.sn[2 * k + 1] : -t.sn[2 * k + 1];
      r[k] = pack_bf16x2(rot_sum(bf_lo(own[k]), t.cs[2 * k], bf_lo(o), s0),
                         rot_sum(bf_hi(own[k]), t.cs[2 * k + 1], bf_hi(o), s1));
    }
  }
  return t.turn ? make_uint4(r[0], r[1], r[2], r[3]) : x;
}

// Positions of row t on every axis that has pairs; false when one of them is outside the table.
__device__ __forceinline__ bool row_positions(const RopeArgs& R, int64_t t, int64_t p, int (&pos)[kRopeAxes]) {
  bool ok = true;
#pragma unroll
  for (int a = 0; a < kRopeAxes; ++a) {
    pos[a] = 0;
    const int begin = a > 0 ? R.sec_end[a - 1] : 0;
    if (a < R.axes && R.sec_end[a] > begin) {
      const int64_t v = R.pos ? (int64_t)R.pos[a * R.pos_stride + t] : p;
      ok = ok && v >= 0 && v < R.P;
      pos[a] = ok ? (int)v : 0;
    }
  }
  return ok;
}

constexpr int kRopeUnroll = 4;  // heads of one lane in flight

// One warp: row t, 32 / LPH * kRopeUnroll heads.
template <int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads) sdpa_rope_kernel(RopeRowsArgs A) {
  constexpr int LPH = D / 8, HPP = 32 / LPH, HPW = HPP * kRopeUnroll;
  const int lane = threadIdx.x & 31, c = lane % LPH;
  const int64_t blocks = (A.H + HPW - 1) / HPW;
  const int64_t n = A.T * blocks, stride = (int64_t)gridDim.x * (kRopeThreads / 32);
  for (int64_t w = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 5; w < n; w += stride) {
    const int64_t t = udiv(w, blocks);
    const int h0 = (int)(w - t * blocks) * HPW + lane / LPH;
    uint4 x[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u)
      if (h0 + u * HPP < A.H)
        x[u] = *reinterpret_cast<const uint4*>(A.x + t * A.x_rs + (int64_t)(h0 + u * HPP) * A.x_hs + 8 * c);
      else
        x[u] = make_uint4(0, 0, 0, 0);
    int pos[kRopeAxes];
    const bool ok = row_positions(A.r, t, 0, pos);
    if (!ok && h0 == 0 && c == 0 && A.status_dev) atomicOr(A.status_dev, SDPA_ROPE_BAD_POS);
    LaneTurn lt;
    lane_turn<IL>(A.r, pos, c, lane, &lt);
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      uint4 y = turn8<IL>(x[u], lt);
      if (!ok) y = make_uint4(0, 0, 0, 0);
      if (h0 + u * HPP < A.H)
        *reinterpret_cast<uint4*>(A.out + t * A.o_rs + (int64_t)(h0 + u * HPP) * A.o_hs + 8 * c) = y;
    }
  }
}

// ------------------------------------------------------------------- rows of a segment table

// A CTA's packed rows [t0, t0 + n): each row's segment, found by every thread looking at the
// segments in turn.  A row is live when exactly one valid segment holds it and that segment shares
// no packed row with another valid one, anywhere.
struct RowTable {
  int owner[kStepRows];
  int dead[kStepRows];
  int4 seg[kStepRows];  // the owner's entry
};

__device__ __forceinline__ void find_rows(const StepArgs& A, int64_t t0, int n, RowTable* s) {
  for (int r = threadIdx.x; r < n; r += blockDim.x) {
    s->owner[r] = -1;
    s->dead[r] = 0;
  }
  __syncthreads();
  auto load = [&](int i, int4* g) -> int32_t {
    *g = __ldg(reinterpret_cast<const int4*>(A.seq_info) + i);
    const int window = A.seg_mode ? __ldg(A.seg_mode + 2 * i + 1) : A.window;
    return segment_bits(g->x, g->y, g->z, g->w, A.T, A.rows, A.cols, window);
  };
  int32_t bits = 0;
  for (int i = threadIdx.x; i < A.S; i += blockDim.x) {
    int4 g;
    const int32_t b = load(i, &g);
    bits |= b;
    if (b || g.y <= 0) continue;
    const int a = (int)max((int64_t)0, (int64_t)g.x - t0), e = (int)min((int64_t)n, (int64_t)g.x + g.y - t0);
    for (int r = a; r < e; ++r) {
      if (atomicCAS(&s->owner[r], -1, i) == -1)
        s->seg[r] = g;
      else
        s->dead[r] = 1;
    }
  }
  if (blockIdx.x == 0 && bits && A.status_dev) atomicOr(A.status_dev, bits);
  __syncthreads();
  // whether another valid segment meets an owner outside these rows
  for (int i = threadIdx.x; i < A.S; i += blockDim.x) {
    int4 g;
    if (load(i, &g) || g.y <= 0) continue;
    for (int r = 0; r < n; ++r) {
      const int o = s->owner[r];
      if (o < 0 || o == i) continue;
      const int4 m = s->seg[r];
      if (max(m.x, g.x) < min(m.x + m.y, g.x + g.y)) s->dead[r] = 1;
    }
  }
  __syncthreads();
  for (int r = threadIdx.x; r < n; r += blockDim.x)
    if (s->dead[r] && A.status_dev) atomicOr(A.status_dev, SDPA_SEG_OVERLAP);
}

// Position of row t0 + r in its sequence, or -1 when no live segment holds it (or it has none).
__device__ __forceinline__ int64_t row_place(const RowTable* s, int64_t t0, int r, int* col) {
  if (s->owner[r] < 0 || s->dead[r]) return -1;
  const int4 g = s->seg[r];
  *col = g.z;
  return (int64_t)g.w - g.y + (t0 + r - g.x);
}

// Largest magnitude of a lane's 8 bf16 values (NaN counts as 0), over the 4 lanes of a scale group.
__device__ __forceinline__ float group_amax(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(bf_lo(w[k])), fabsf(bf_hi(w[k]))));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
__device__ __forceinline__ uint32_t codes8(const uint4& x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) c |= (q4_code(bf_lo(w[k]), s) | q4_code(bf_hi(w[k]), s) << 4) << (8 * k);
  return c;
}

// A step's rows: queries rotated into q_out, keys rotated and values as they are into the store.
// A CTA takes `cr` packed rows; a warp takes a row and 32 / LPH * kRopeUnroll heads of its q, k or v.
template <int D, bool IL, bool Q4>
__global__ void __launch_bounds__(kRopeThreads) sdpa_rope_append_kernel(StepArgs A) {
  __shared__ RowTable s_rows;
  constexpr int LPH = D / 8, HPP = 32 / LPH, HPW = HPP * kRopeUnroll;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LPH, hs = lane / LPH;
  const int64_t t0 = (int64_t)blockIdx.x * A.cr;
  const int n = (int)min((int64_t)A.cr, A.T - t0);
  find_rows(A, t0, n, &s_rows);

  const int qb = (A.Hq + HPW - 1) / HPW, kb = (A.Hkv + HPW - 1) / HPW, per = qb + 2 * kb;
  for (int w = warp; w < n * per; w += kRopeThreads / 32) {
    const int r = w / per, b = w - r * per;
    const int64_t t = t0 + r;
    const int what = b < qb ? 0 : b < qb + kb ? 1 : 2;  // q, k, v
    const int h0 = (b - (what == 0 ? 0 : what == 1 ? qb : qb + kb)) * HPW + hs;
    const int H = what == 0 ? A.Hq : A.Hkv;
    const __nv_bfloat16* src = what == 0 ? A.q : what == 1 ? A.k : A.v;
    const int64_t rs = what == 0 ? A.q_rs : what == 1 ? A.k_rs : A.v_rs;
    const int64_t xs = what == 0 ? A.q_hs : what == 1 ? A.k_hs : A.v_hs;
    uint4 x[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      if (h0 + u * HPP < H)
        x[u] = *reinterpret_cast<const uint4*>(src + t * rs + (int64_t)(h0 + u * HPP) * xs + 8 * c);
    }
    int col = 0;
    const int64_t p = row_place(&s_rows, t0, r, &col);
    int pos[kRopeAxes];
    const bool in = p < 0 || row_positions(A.r, t, p, pos);
    const bool ok = p >= 0 && in;
    if (!in && what == 0 && h0 == 0 && c == 0 && A.status_dev) atomicOr(A.status_dev, SDPA_ROPE_BAD_POS);
    if (what > 0 && !ok) continue;  // nothing of the row is kept (the warp has one row)
    if (what < 2 && ok) {
      LaneTurn lt;
      lane_turn<IL>(A.r, pos, c, lane, &lt);
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u) x[u] = turn8<IL>(x[u], lt);
    }
    if (what == 0) {
#pragma unroll
      for (int u = 0; u < kRopeUnroll; ++u)
        if (h0 + u * HPP < H)
          *reinterpret_cast<uint4*>(A.q_out + t * A.o_rs + (int64_t)(h0 + u * HPP) * A.o_hs + 8 * c) =
              ok ? x[u] : make_uint4(0, 0, 0, 0);
      continue;
    }
    const int64_t row = (uint32_t)p % (uint32_t)A.rows;  // both below 2^31
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int h = h0 + u * HPP;
      if constexpr (Q4) {
        const uint32_t sb = q4_scale_byte(group_amax(x[u]));
        if (h < H) {
          const int64_t cell = ((int64_t)col * A.Hkv + h) * A.rows + row;
          uint8_t* codes = what == 1 ? A.q4.kc : A.q4.vc;
          uint8_t* scales = what == 1 ? A.q4.ks : A.q4.vs;
          *reinterpret_cast<uint32_t*>(codes + cell * (D / 2) + 4 * c) = codes8(x[u], q4_scale(sb));
          if (c % 4 == 0) scales[cell * (D / kQ4Group) + c / 4] = (uint8_t)sb;
        }
      } else if (h < H) {
        __nv_bfloat16* st = what == 1 ? A.k_store : A.v_store;
        *reinterpret_cast<uint4*>(st + ((row * A.cols + col) * A.Hkv + h) * (int64_t)D + 8 * c) = x[u];
      }
    }
  }
}

// The rows of a segment table read back from a 4-bit store as bf16 (exact), rows that no live
// segment holds and rows before a sequence's beginning as 0.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) sdpa_q4_unpack_kernel(StepArgs A) {
  __shared__ RowTable s_rows;
  constexpr int LPH = D / 8;
  const int64_t t0 = (int64_t)blockIdx.x * A.cr;
  const int n = (int)min((int64_t)A.cr, A.T - t0);
  find_rows(A, t0, n, &s_rows);
  const int per = A.Hkv * LPH;  // chunks of 8 dims of a row
  for (int w = threadIdx.x; w < n * per; w += kRopeThreads) {
    const int r = w / per, x = w - r * per, h = x / LPH, c = x % LPH;
    int col = 0;
    const int64_t p = row_place(&s_rows, t0, r, &col);
    const int64_t cell = p < 0 ? 0 : ((int64_t)col * A.Hkv + h) * A.rows + (uint32_t)p % (uint32_t)A.rows;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint4 y = make_uint4(0, 0, 0, 0);
      if (p >= 0) y = q4_words8(*reinterpret_cast<const uint32_t*>((v ? A.q4.vc : A.q4.kc) + cell * (D / 2) + 4 * c),
                                (v ? A.q4.vs : A.q4.ks)[cell * (D / kQ4Group) + c / 4]);
      __nv_bfloat16* dst = v ? A.v_out : A.k_out;
      *reinterpret_cast<uint4*>(dst + (t0 + r) * A.o_rs + (int64_t)h * A.o_hs + 8 * c) = y;
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
int rope_heads_per_warp(int D) { return 32 / (D / 8) * kRopeUnroll; }

}  // namespace sdpa
