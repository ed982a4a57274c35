// step.cuh - device code that the rotary kernels share (rope.cu, q8_step.cu): pairs of a row turned, and a
// step's packed rows looked up in its segment table.
#pragma once

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

// ------------------------------------------------------------------- rows of a segment table

// A CTA's packed rows [t0, t0 + n): each row's segment, found by every thread looking at the
// segments in turn.  A row is live when exactly one valid segment holds it and that segment shares
// no packed row with another valid one, anywhere.
struct RowTable {
  int owner[kStepRows];
  int dead[kStepRows];
  int shared[kStepRows]; // BLOCKS: another valid segment writes to a block that the row's segment writes to
  int4 seg[kStepRows];   // the owner's entry
  int2 cell[kStepRows];  // (store row, column), or (-1, 0): nothing of the row is kept
  int pos[kStepRows][kRopeAxes];
};

// Entry i of the table, and its status bits.
__device__ __forceinline__ int32_t load_entry(const StepArgs& A, int i, int4* g) {
  *g = __ldg(reinterpret_cast<const int4*>(A.seq_info) + i);
  const int window = A.seg_mode ? __ldg(A.seg_mode + 2 * i + 1) : A.window;
  return segment_bits(g->x, g->y, g->z, g->w, A.T, A.rows, A.cols, window);
}
// Whether two segments share a packed row.
__device__ __forceinline__ bool rows_meet(const int4& a, const int4& b) {
  return max(a.x, b.x) < min(a.x + a.y, b.x + b.y);
}

template <bool BLOCKS>
__device__ __forceinline__ void find_rows(const StepArgs& A, int64_t t0, int n, RowTable* s, bool report) {
  auto load = [&](int i, int4* g) -> int32_t { return load_entry(A, i, g); };
  const int tid = threadIdx.x;
  int4 g0 = make_int4(0, 0, 0, 0);  // a thread keeps its first segment
  int32_t bits0 = 0;
  if (tid < A.S) bits0 = load(tid, &g0);
  if (tid < n) {
    s->owner[tid] = -1;
    s->dead[tid] = 0;
    if (BLOCKS) s->shared[tid] = 0;
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
  if (report && bits && A.status_dev) atomicOr(A.status_dev, bits);
  __syncthreads();
  if (A.S <= 1) return;
  // whether another valid segment meets an owner outside these rows
  for (int i = tid; i < A.S; i += kRopeThreads) {
    int4 g = g0;
    const int32_t b = i == tid ? bits0 : load(i, &g);
    if (b || g.y <= 0) continue;
    bool column = false;
    for (int r = 0; r < n; ++r) {
      const int o = s->owner[r];
      if (o < 0 || o == i) continue;
      const int4 m = s->seg[r];
      if (rows_meet(m, g)) s->dead[r] = 1;
      column |= m.z == g.z;
    }
    if (!BLOCKS || !column) continue;
    for (int r = 0; r < n; ++r) {
      const int o = s->owner[r];
      if (o < 0 || o == i) continue;
      const int4 m = s->seg[r];
      if (m.z == g.z && blocks_meet(m.y, m.w, g.y, g.w, A.rows)) s->shared[r] = 1;
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

__device__ __forceinline__ float amax8(const uint32_t (&w)[4]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(bf_lo(w[k])), fabsf(bf_hi(w[k]))));
  return m;
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

// A step's rows: queries rotated into q_out and (KV) keys and values handed to `store`, the keys as they are
// to be rotated.  The work is a line of passes (32 / (D / 16) heads each), a row's being those of q, then k, then v;
// block `block` takes `per` of them in order, at most kStepRows rows at a time, its warps even shares of
// those.  Two passes are always on their way, the first ones while the rows' segments are looked
// up, and the angles of a warp's next row while it is at one.
template <int D, bool IL, bool KV, class Store>
__device__ __forceinline__ void step_passes(const StepArgs& A, int block, RowTable& s_rows, float2 (*s_angles)[D / 2],
                                            Store store) {
  constexpr int LPH = D / 16, HPP = 32 / LPH, kWarps = kRopeThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hs = lane / LPH;
  const LaneDims<IL> ld(A.r.half, lane % LPH);
  const int j0 = ld.turn ? ld.j0 : 0;
  const int pq = (A.Hq + HPP - 1) / HPP, pk = KV ? (A.Hkv + HPP - 1) / HPP : 0, passes = pq + 2 * pk;
  const int64_t f_end = min((int64_t)(block + 1) * A.per, A.T * passes);

  // passes [fa, fb) of the line, rows [t0, t0 + n), and this warp's share [wa, wb) counted from row t0
  for (int64_t fa = (int64_t)block * A.per; fa < f_end;) {
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
    find_rows<false>(A, t0, n, &s_rows, block == 0);
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
        store(y, ld, an, what == 1, h, lane, cell);
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

}  // namespace sdpa
