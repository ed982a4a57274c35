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

// A pair turned, the quick way: r = fma(a, c, b s) is off by at most 2^-24 of |r| + |b s|.  Rounding to
// fp32 and to bf16 are both monotone, so where r - E and r + E (E a little more than that, each end
// rounded once) come to the same bf16, the exact value does too.  Where they do not (one value in
// some 2^14, or infinities) *unsure is set and the caller takes rot_sum.
struct Ends {
  float lo, hi;
};
__device__ __forceinline__ Ends rot_ends(float a, float c, float b, float s) {
  constexpr float k = 0x1.001p-24f;
  const float q = b * s, r = fmaf(a, c, q);
  const float t = fabsf(q) + fabsf(r);
  return {fmaf(t, -k, r), fmaf(t, k, r)};
}
__device__ __forceinline__ uint32_t pack_ends(const Ends& x, const Ends& y, uint32_t* unsure) {
  const uint32_t lo = pack_bf16x2(x.lo, y.lo);
  *unsure |= lo ^ pack_bf16x2(x.hi, y.hi);
  return lo;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The 16 dims of a head that a lane takes: 8 from da on and 8 from db on.  The lanes of a head are
// D / 16; the first rot_dims / 16 of them turn 8 pairs each, the others pass 16 dims on.
template <bool IL>
struct LaneDims {
  int da, db, j0;  // j0: the first of the lane's pairs
  bool turn;
  __device__ __forceinline__ LaneDims(int half, int i) {
    turn = 8 * i < half;
    j0 = 8 * i;
    da = IL || !turn ? 16 * i : 8 * i;
    db = IL || !turn ? 16 * i + 8 : half + 8 * i;
  }
};
struct Row16 {
  uint4 a, b;
};

struct Angles {
  float cs[8], sn[8];  // of a lane's pairs
};

// The angles of a row whose positions are pos[axis]: the warp fetches each pair's once (a pair's axis
// is where its section lies), and the lanes take theirs from shared memory.
struct PairAngles {
  float2 v[4];  // pairs lane, lane + 32, ... of the row's (at most 128)
};
template <int D>
__device__ __forceinline__ void fetch_angles(const RopeArgs& R, const int (&pos)[kRopeAxes], int lane, PairAngles* f) {
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const int j = lane + 32 * k;
    if (j < R.half) {
      int p = pos[0];
      if (R.axes > 1) {
#pragma unroll
        for (int a = 1; a < kRopeAxes; ++a) p = j >= R.sec_end[a - 1] ? pos[a] : p;
      }
      f->v[k] = __ldg(R.table + (uint32_t)(p * R.half + j));  // below 2^31 (checked on the host)
    }
  }
}
// sh: the warp's own D / 2 pairs.  Every lane calls it.
template <int D>
__device__ __forceinline__ void share_angles(const RopeArgs& R, const PairAngles& f, int j0, int lane, float2* sh,
                                             Angles* t) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    const int j = lane + 32 * k;
    if (j < R.half) sh[j] = R.inverse ? make_float2(f.v[k].x, -f.v[k].y) : f.v[k];
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = reinterpret_cast<const float4*>(sh + j0)[k];
    t->cs[2 * k] = v.x; t->sn[2 * k] = v.y;
    t->cs[2 * k + 1] = v.z; t->sn[2 * k + 1] = v.w;
  }
}

// Turns a lane's 8 pairs: (a, b) of pair k are dims da + k and db + k, or 2k and 2k + 1 of the 16.
template <bool IL, bool EXACT>
__device__ __forceinline__ void turn16(Row16* x, const Angles& t) {
  const uint32_t a[4] = {x->a.x, x->a.y, x->a.z, x->a.w}, b[4] = {x->b.x, x->b.y, x->b.z, x->b.w};
  uint32_t ra[4], rb[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // pairs (u, v) at angle i and (w, z) at angle j
    const float u = bf_lo(a[k]), v = IL ? bf_hi(a[k]) : bf_lo(b[k]);
    const float w = IL ? bf_lo(b[k]) : bf_hi(a[k]), z = bf_hi(b[k]);
    const int i = IL ? k : 2 * k, j = IL ? 4 + k : 2 * k + 1;
    if constexpr (!EXACT) {
      const float u0 = fmaf(u, t.cs[i], -(v * t.sn[i])), v0 = fmaf(v, t.cs[i], u * t.sn[i]);
      const float w0 = fmaf(w, t.cs[j], -(z * t.sn[j])), z0 = fmaf(z, t.cs[j], w * t.sn[j]);
      ra[k] = pack_bf16x2(u0, IL ? v0 : w0);
      rb[k] = pack_bf16x2(IL ? w0 : v0, z0);
      continue;
    }
    const Ends u1 = rot_ends(u, t.cs[i], v, -t.sn[i]), v1 = rot_ends(v, t.cs[i], u, t.sn[i]);
    const Ends w1 = rot_ends(w, t.cs[j], z, -t.sn[j]), z1 = rot_ends(z, t.cs[j], w, t.sn[j]);
    uint32_t unsure = 0;
    ra[k] = pack_ends(u1, IL ? v1 : w1, &unsure);
    rb[k] = pack_ends(IL ? w1 : v1, z1, &unsure);
    if (unsure) {
      const float u2 = rot_sum(u, t.cs[i], v, -t.sn[i]), v2 = rot_sum(v, t.cs[i], u, t.sn[i]);
      const float w2 = rot_sum(w, t.cs[j], z, -t.sn[j]), z2 = rot_sum(z, t.cs[j], w, t.sn[j]);
      ra[k] = pack_bf16x2(u2, IL ? v2 : w2);
      rb[k] = pack_bf16x2(IL ? w2 : v2, z2);
    }
  }
  x->a = make_uint4(ra[0], ra[1], ra[2], ra[3]);
  x->b = make_uint4(rb[0], rb[1], rb[2], rb[3]);
}

__device__ __forceinline__ uint4 ldg16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void stg16(__nv_bfloat16* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

// Positions of row t on every axis (p where none are given).
__device__ __forceinline__ void fetch_positions(const RopeArgs& R, int64_t t, int p, int (&pos)[kRopeAxes]) {
#pragma unroll
  for (int a = 0; a < kRopeAxes; ++a) {
    pos[a] = p;
    if (R.pos && a < R.axes) pos[a] = __ldg(R.pos + a * R.pos_stride + t);
  }
}
// Whether those of the axes that have pairs lie in the table; the others, and all when one does not,
// are set to a row that does.
__device__ __forceinline__ bool check_positions(const RopeArgs& R, int (&pos)[kRopeAxes]) {
  bool ok = true;
#pragma unroll
  for (int a = 0; a < kRopeAxes; ++a) {
    const bool used = a < R.axes && R.sec_end[a] > (a > 0 ? R.sec_end[a - 1] : 0);
    const bool in = (uint32_t)pos[a] < (uint32_t)R.P;
    ok = ok && (in || !used);
    pos[a] = in ? pos[a] : 0;
  }
  return ok;
}

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

// ------------------------------------------------------------------- rows of a segment table

// A CTA's packed rows [t0, t0 + n): each row's segment, found by every thread looking at the
// segments in turn.  A row is live when exactly one valid segment holds it and that segment shares
// no packed row with another valid one, anywhere.
struct RowTable {
  int owner[kStepRows];
  int dead[kStepRows];
  int4 seg[kStepRows];   // the owner's entry
  int2 cell[kStepRows];  // (store row, column), or (-1, 0): nothing of the row is kept
  int pos[kStepRows][kRopeAxes];
};

__device__ __forceinline__ void find_rows(const StepArgs& A, int64_t t0, int n, RowTable* s) {
  auto load = [&](int i, int4* g) -> int32_t {
    *g = __ldg(reinterpret_cast<const int4*>(A.seq_info) + i);
    const int window = A.seg_mode ? __ldg(A.seg_mode + 2 * i + 1) : A.window;
    return segment_bits(g->x, g->y, g->z, g->w, A.T, A.rows, A.cols, window);
  };
  const int tid = threadIdx.x;
  int4 g0 = make_int4(0, 0, 0, 0);  // a thread keeps its first segment
  int32_t bits0 = 0;
  if (tid < A.S) bits0 = load(tid, &g0);
  if (tid < n) {
    s->owner[tid] = -1;
    s->dead[tid] = 0;
  }
  __syncthreads();
  int32_t bits = 0;
  for (int i = tid; i < A.S; i += kRopeThreads) {
    int4 g = g0;
    const int32_t b = i == tid ? bits0 : load(i, &g);
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
  if (A.S <= 1) return;
  // whether another valid segment meets an owner outside these rows
  for (int i = tid; i < A.S; i += kRopeThreads) {
    int4 g = g0;
    const int32_t b = i == tid ? bits0 : load(i, &g);
    if (b || g.y <= 0) continue;
    for (int r = 0; r < n; ++r) {
      const int o = s->owner[r];
      if (o < 0 || o == i) continue;
      const int4 m = s->seg[r];
      if (max(m.x, g.x) < min(m.x + m.y, g.x + g.y)) s->dead[r] = 1;
    }
  }
  __syncthreads();
  if (tid < n && s->dead[tid] && A.status_dev) atomicOr(A.status_dev, SDPA_SEG_OVERLAP);
}

// Position of row t0 + r in its sequence, or -1 when no live segment holds it (or it has none).
__device__ __forceinline__ int64_t row_place(const RowTable* s, int64_t t0, int r, int* col) {
  if (s->owner[r] < 0 || s->dead[r]) return -1;
  const int4 g = s->seg[r];
  *col = g.z;
  return (int64_t)g.w - g.y + (t0 + r - g.x);
}

// A lane's 8 bf16 values with NaN as 0, clamped to what the largest scale holds (7 * 1920).
__device__ __forceinline__ uint32_t q4_storable(uint32_t w) {
  __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w);
  const uint32_t clean = w & __heq2_mask(v, v);
  v = *reinterpret_cast<const __nv_bfloat162*>(&clean);
  v = __hmin2(__hmax2(v, __float2bfloat162_rn(-13440.f)), __float2bfloat162_rn(13440.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float amax8(const uint32_t (&w)[4]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(bf_lo(w[k])), fabsf(bf_hi(w[k]))));
  return m;
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

// The rest of what the warps need of rows [t0, t0 + n): where each goes, and its positions.
__device__ __forceinline__ void place_rows(const StepArgs& A, int64_t t0, int n, RowTable* s) {
  const int r = threadIdx.x;
  if (r < n) {
    int col = 0;
    const int64_t place = row_place(s, t0, r, &col);
    int pos[kRopeAxes] = {0, 0, 0, 0};
    if (place >= 0) fetch_positions(A.r, t0 + r, (int)place, pos);
    const bool in = check_positions(A.r, pos);
    if (!in && A.status_dev) atomicOr(A.status_dev, SDPA_ROPE_BAD_POS);
    // (positions and rows are below 2^31)
    s->cell[r] = place >= 0 && in ? make_int2((int)((uint32_t)place % (uint32_t)A.rows), col) : make_int2(-1, 0);
#pragma unroll
    for (int a = 0; a < kRopeAxes; ++a) s->pos[r][a] = pos[a];
  }
  __syncthreads();
}

// A step's rows: queries rotated into q_out, keys rotated and values as they are into the store.
// The work is a line of passes (32 / (D / 16) heads each), a row's being those of q, then k, then v;
// a CTA takes `per` of them in order, at most kStepRows rows at a time, its warps even shares of
// those.  Two passes are always on their way, the first ones while the rows' segments are looked
// up, and the angles of a warp's next row while it is at one.
template <int D, bool IL, bool Q4>
__global__ void __launch_bounds__(kRopeThreads, 3) sdpa_rope_append_kernel(StepArgs A) {
  constexpr int LPH = D / 16, HPP = 32 / LPH, kWarps = kRopeThreads / 32;
  __shared__ RowTable s_rows;
  __shared__ __align__(16) float2 s_angles[kWarps][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hs = lane / LPH;
  const LaneDims<IL> ld(A.r.half, lane % LPH);
  const int j0 = ld.turn ? ld.j0 : 0;
  const int pq = (A.Hq + HPP - 1) / HPP, pk = (A.Hkv + HPP - 1) / HPP, passes = pq + 2 * pk;
  const int64_t f_end = min((int64_t)(blockIdx.x + 1) * A.per, A.T * passes);

  // passes [fa, fb) of the line, rows [t0, t0 + n), and this warp's share [wa, wb) counted from row t0
  for (int64_t fa = (int64_t)blockIdx.x * A.per; fa < f_end;) {
    const int64_t t0 = udiv(fa, passes);
    const int64_t fb = min(f_end, (t0 + kStepRows) * passes);
    const int n = (int)udiv(fb - 1, passes) - (int)t0 + 1;
    const int off = (int)(fa - t0 * passes), len = (int)(fb - fa);
    const int wa = off + len * warp / kWarps, wb = off + len * (warp + 1) / kWarps;
    fa = fb;

    Row16 x[2];
    int lr = wa / passes, lp = wa - lr * passes;  // the next pass to load
    auto load = [&](Row16* y) {
      y->a = y->b = make_uint4(0, 0, 0, 0);
      if (lr * passes + lp >= wb) return;
      const int what = lp < pq ? 0 : lp < pq + pk ? 1 : 2;
      const int h = (lp - (what == 0 ? 0 : what == 1 ? pq : pq + pk)) * HPP + hs;
      if (h < (what == 0 ? A.Hq : A.Hkv)) {
        const int64_t t = t0 + lr;
        const __nv_bfloat16* z = what == 0 ? A.q + t * A.q_rs + (int64_t)h * A.q_hs
                                 : what == 1 ? A.k + t * A.k_rs + (int64_t)h * A.k_hs
                                             : A.v + t * A.v_rs + (int64_t)h * A.v_hs;
        y->a = ldg16(z + ld.da);
        y->b = ldg16(z + ld.db);
      }
      if (++lp == passes) {
        lp = 0;
        ++lr;
      }
    };
    int r = lr, p = lp;  // the pass at hand
    load(&x[0]);
    load(&x[1]);
    find_rows(A, t0, n, &s_rows);
    place_rows(A, t0, n, &s_rows);

    if (wa < wb) {
      PairAngles pa;
      fetch_angles<D>(A.r, s_rows.pos[r], lane, &pa);
      Angles an;
      int2 cell;
      auto enter_row = [&]() {
        cell = s_rows.cell[r];
        share_angles<D>(A.r, pa, j0, lane, s_angles[warp], &an);
        if ((r + 1) * passes < wb) fetch_angles<D>(A.r, s_rows.pos[r + 1], lane, &pa);
      };
      enter_row();
      auto work = [&](Row16& y) {
        const int what = p < pq ? 0 : p < pq + pk ? 1 : 2;
        const int h = (p - (what == 0 ? 0 : what == 1 ? pq : pq + pk)) * HPP + hs;
        const bool ok = cell.x >= 0;
        if (what == 0) {
          if (ld.turn) turn16<IL, false>(&y, an);
          if (!ok) y.a = y.b = make_uint4(0, 0, 0, 0);
          if (h < A.Hq) {
            __nv_bfloat16* z = A.q_out + (t0 + r) * A.o_rs + (int64_t)h * A.o_hs;
            stg16(z + ld.da, y.a);
            stg16(z + ld.db, y.b);
          }
          return;
        }
        if (!ok) return;  // (the warp has one row)
        if (what == 1 && ld.turn) turn16<IL, true>(&y, an);
        if constexpr (Q4) {
          const uint32_t ca[4] = {q4_storable(y.a.x), q4_storable(y.a.y), q4_storable(y.a.z), q4_storable(y.a.w)};
          const uint32_t cb[4] = {q4_storable(y.b.x), q4_storable(y.b.y), q4_storable(y.b.z), q4_storable(y.b.w)};
          float ma = amax8(ca), mb = amax8(cb);
          group_amax<LPH>(&ma, &mb, IL, A.r.half, lane);
          const uint32_t ba = q4_scale_byte(ma), bb = q4_scale_byte(mb);
          if (h < A.Hkv) {
            const int64_t at = ((int64_t)cell.y * A.Hkv + h) * A.rows + cell.x;
            uint8_t* codes = (what == 1 ? A.q4.kc : A.q4.vc) + at * (D / 2);
            uint8_t* scales = (what == 1 ? A.q4.ks : A.q4.vs) + at * (D / kQ4Group);
            *reinterpret_cast<uint32_t*>(codes + ld.da / 2) = codes8(ca, ba);
            *reinterpret_cast<uint32_t*>(codes + ld.db / 2) = codes8(cb, bb);
            if (ld.da % kQ4Group == 0) scales[ld.da / kQ4Group] = (uint8_t)ba;
            if (ld.db % kQ4Group == 0) scales[ld.db / kQ4Group] = (uint8_t)bb;
          }
        } else if (h < A.Hkv) {
          __nv_bfloat16* z =
              (what == 1 ? A.k_store : A.v_store) + (((int64_t)cell.x * A.cols + cell.y) * A.Hkv + h) * D;
          stg16(z + ld.da, y.a);
          stg16(z + ld.db, y.b);
        }
      };
      for (int f = wa; f < wb; f += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (f + u >= wb) break;
          work(x[u]);
          load(&x[u]);
          if (++p == passes && f + u + 1 < wb) {
            p = 0;
            ++r;
            enter_row();
          }
        }
      }
    }
    if (fa < f_end) __syncthreads();  // the rows' records are written again
  }
}

// The rows of a segment table read back from a 4-bit store as bf16 (exact), rows that no live
// segment holds and rows before a sequence's beginning as 0.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) sdpa_q4_unpack_kernel(StepArgs A) {
  __shared__ RowTable s_rows;
  constexpr int LPH = D / 8, U = 4;
  const int64_t t0 = (int64_t)blockIdx.x * A.cr;
  const int n = (int)min((int64_t)A.cr, A.T - t0);
  find_rows(A, t0, n, &s_rows);
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
