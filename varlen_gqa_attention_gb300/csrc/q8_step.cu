// q8_step.cu - a step's rows rotated and written into the 8-bit column store, and rows read back from it.
//
// A block of 16 rows of a head shares a scale, so a block is coded as a whole: a warp takes one block of one head
// of K or of V, holds its new rows (keys rotated exactly to bf16, as for the 4-bit store: see rope.cu) and the
// rows that it keeps, takes their largest magnitude, and writes the new rows' codes, and the others' again if the
// scale changed.  Nothing is read twice, and nothing is exchanged between warps.
//   * A CTA looks at a run of packed rows for those that are the first of their block in a segment, and takes
//     these blocks one after another: their rows' cells and angles in shared memory, then a warp a (head, K or V).
//   * A row that the step does not write is kept if it holds a position from before the step: the block's earlier
//     rows, and on a ring that has wrapped the later ones too.  What else lies in the block (a former sequence's
//     rows) counts for nothing and keeps its bytes.
//   * A step that fills a whole ring may come back to the block it began in; the block's first visit then takes
//     the rows of both.
//   * A block that several segments write to is coded by the first of them, with the rows of all.
// The queries are rotated by CTAs of their own in the same launch.
//
// What bounds it: 4093 tokens of 32/8 heads, D = 128, three position axes, take 23.2 us (4.0 TB/s; a loop over the same
// buffers): 11.6 the queries alone, 2.9 more the look-up of rows and angles, 8.5 the blocks, of which the rotation
// is 2; no pipe is full (1.6 instructions a cycle at 24 warps an SM).  Two CTAs for a block's heads (27.8 us), the blocks'
// CTAs behind the queries' (34.2), the queries' rest given to the blocks' CTAs so that all make one wave (31 to 34), a
// block's queries rotated by its own CTA by the angles it has (31), and rows in shared memory instead of registers, with
// loops that are not unrolled (24.3), were all slower.  32 single tokens: 5.1 us, the chain table - row and block - codes.
// The read-back: 57025 tokens of 8 heads 61.8 us, 5.7 TB/s (0.84 of the measured copy rate), two thirds of it writes.
#include "q8.cuh"
#include "step.cuh"

namespace sdpa {

// A lane's 8 bf16 values with NaN as 0, clamped to what the largest scale holds (127 * 512).
__device__ __forceinline__ uint32_t q8_storable(uint32_t w) {
  __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w);
  const uint32_t clean = w & __heq2_mask(v, v);
  v = *reinterpret_cast<const __nv_bfloat162*>(&clean);
  v = __hmin2(__hmax2(v, __float2bfloat162_rn(-65024.f)), __float2bfloat162_rn(65024.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The low byte of round(v): adding 1.5 * 2^23 rounds (halves to even) and leaves the integer's two's complement in
// the low bits.  A code is that with its top bit turned.
__device__ __forceinline__ uint32_t q8_low(float v) { return __float_as_uint(v + 12582912.f); }
__device__ __forceinline__ uint32_t q8_codes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410) ^ 0x80808080u;
}
// The codes of 8 bf16 values, inv being 1 / s (a power of two: the product is exact).
__device__ __forceinline__ uint2 q8_codes8(const uint4& w, float inv) {
  return make_uint2(q8_codes4(q8_low(bf_lo(w.x) * inv), q8_low(bf_hi(w.x) * inv), q8_low(bf_lo(w.y) * inv),
                              q8_low(bf_hi(w.y) * inv)),
                    q8_codes4(q8_low(bf_lo(w.z) * inv), q8_low(bf_hi(w.z) * inv), q8_low(bf_lo(w.w) * inv),
                              q8_low(bf_hi(w.w) * inv)));
}
__device__ __forceinline__ float q8_int(uint32_t w, int k) { return (float)(int)((w >> (8 * k) & 255u) - 128); }
// A word of codes under a scale `ratio` (s before / s after) times as coarse.
__device__ __forceinline__ uint32_t q8_again(uint32_t w, float ratio) {
  return q8_codes4(q8_low(q8_int(w, 0) * ratio), q8_low(q8_int(w, 1) * ratio), q8_low(q8_int(w, 2) * ratio),
                   q8_low(q8_int(w, 3) * ratio));
}
__device__ __forceinline__ float q8_amax4(uint32_t w) {
  return fmaxf(fmaxf(fabsf(q8_int(w, 0)), fabsf(q8_int(w, 1))), fmaxf(fabsf(q8_int(w, 2)), fabsf(q8_int(w, 3))));
}
// Largest magnitudes of bf16 pairs, as bit patterns (they are ordered as the magnitudes are, NaN beyond infinity).
__device__ __forceinline__ uint32_t pair_amax(uint32_t m, const uint4& w) {
  m = __vmaxu2(m, __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu));
  return __vmaxu2(m, __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
}
constexpr uint32_t kQ8Most = 0x477Eu;  // 65024 in bf16

// What the warps need of a run's blocks: where a block lies (its first store row, its column), where its rows come
// from (a packed row, kKept or kNone), and whether any comes from a packed row.
constexpr int kKept = -1, kNone = -2;
struct BlockRows {
  int2 at[kStepRows];
  int fresh[kStepRows];
  int src[kStepRows][kPackedRows];
  int pos[kStepRows][kPackedRows][kRopeAxes];
  __device__ __forceinline__ void put(int f, int row, int s, const int (&p)[kRopeAxes]) {
    src[f][row] = s;
#pragma unroll
    for (int a = 0; a < kRopeAxes; ++a) pos[f][row][a] = p[a];
  }
};

// Where a live segment's rows leave a store row of its column: the packed row that is written there (and that row's
// positions), kKept, or kNone.
__device__ __forceinline__ int block_row(const StepArgs& A, const int4& g, int64_t row, int (&pos)[kRopeAxes]) {
  const int64_t last = (int64_t)g.w - 1, begin = max((int64_t)g.w - g.y, (int64_t)0);
  if (row > last) return kNone;
  const int64_t p = last - (uint32_t)(last - row) % (uint32_t)A.rows;  // the last position that the row may hold
  if (p < begin) return kKept;
  const int src = (int)(g.x + (p - ((int64_t)g.w - g.y)));
  fetch_positions(A.r, src, (int)p, pos);
  if (check_positions(A.r, pos)) return src;
  return p - A.rows >= 0 ? kKept : kNone;  // nothing of the row is written
}

// The live segments that write to one block, where one of them is known to share a block with another: the first of
// them, which codes it, and for each row the last one that writes it, and whether any keeps it.  All threads of the CTA
// look at the table together.  A segment is live when no other valid one has packed rows of it, as all are when each
// begins behind the one before; in other tables the thread asks all of them.
struct BlockWriters {
  int first;
  int last[kPackedRows], kept[kPackedRows];
};
__device__ __forceinline__ void find_writers(const StepArgs& A, int col, int64_t brow, BlockWriters& w) {
  if (threadIdx.x < kPackedRows) {
    w.first = INT_MAX;
    w.last[threadIdx.x] = -1;
    w.kept[threadIdx.x] = 0;
  }
  bool mixed = false;
  for (int i = threadIdx.x; i < A.S; i += kRopeThreads) {
    int4 g, o;
    if (load_entry(A, i, &g) || g.y <= 0) continue;
    for (int j = i - 1; j >= 0; --j) {
      if (load_entry(A, j, &o) || o.y <= 0) continue;
      mixed |= o.x + o.y > g.x;
      break;
    }
  }
  mixed = __syncthreads_or(mixed);
  for (int i = threadIdx.x; i < A.S; i += kRopeThreads) {
    int4 g;
    if (load_entry(A, i, &g) || g.y <= 0 || g.z != col) continue;
    if (!runs_meet(block_run(g.y, g.w), {brow / kPackedRows, 1}, A.rows / kPackedRows)) continue;
    bool live = true;
    for (int j = 0; mixed && j < A.S; ++j) {
      int4 o;
      if (load_entry(A, j, &o) == 0 && o.y > 0 && j != i && rows_meet(g, o)) live = false;
    }
    if (!live) continue;
    atomicMin(&w.first, i);
#pragma unroll 1
    for (int c = 0; c < kPackedRows; ++c) {
      int pos[kRopeAxes];
      const int src = block_row(A, g, brow + c, pos);
      if (src >= 0) atomicMax(&w.last[c], i);
      if (src == kKept) w.kept[c] = 1;
    }
  }
  __syncthreads();
}

// The rows of those of a run's blocks that other segments write to as well.  Out of line: as part of the kernel, which has
// next to no tables of this kind, it took the chunks of 4000 rows 2 us of 35.
static __device__ __noinline__ void share_blocks(const StepArgs& A, const RowTable& rows, BlockRows& blocks, BlockWriters& w,
                                                 const int* first, int count) {
  const int lane = threadIdx.x & 31, row = lane % kPackedRows;
  for (int f = 0; f < count; ++f) {
    const int r = first[f];
    if (!rows.shared[r]) continue;
    const int2 at = blocks.at[f];
    find_writers(A, at.y, at.x, w);
    if (threadIdx.x < 32) {
      int src = kNone, pos[kRopeAxes] = {0, 0, 0, 0};
      if (w.first == rows.owner[r]) {  // (else that segment's visit codes the block)
        if (w.last[row] >= 0) {
          int4 g;
          load_entry(A, w.last[row], &g);
          src = block_row(A, g, at.x + row, pos);
        } else if (w.kept[row]) {
          src = kKept;
        }
      }
      const bool fresh = __any_sync(0xffffffffu, src >= 0);
      if (lane < kPackedRows) blocks.put(f, row, src, pos);
      if (lane == 0) blocks.fresh[f] = fresh;
    }
    __syncthreads();
  }
}

template <int D, bool IL>
__device__ __forceinline__ void code_blocks(const StepArgs& A, int block, RowTable& s_rows, BlockRows& s_block,
                                            BlockWriters& s_writers, int (&s_first)[kStepRows], int& s_count, int& s_share,
                                            float2 (*s_angles)[D / 2]) {
  constexpr int LPH = D / 16, RPP = 32 / LPH, U = kPackedRows / RPP, kWarps = kRopeThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, li = lane % LPH, ls = lane / LPH;
  const LaneDims<IL> ld(A.r.half, li);
  const int j0 = ld.turn ? ld.j0 : 0;
  const int part = block % A.kv_parts;
  const int64_t t0 = (int64_t)(block / A.kv_parts) * A.cr;
  const int n = (int)min((int64_t)A.cr, A.T - t0);
  // this CTA's heads; items: their keys (whose rotation takes most), then their values, so that the warps' shares are even
  const int ha = A.Hkv * part / A.kv_parts, heads = A.Hkv * (part + 1) / A.kv_parts - ha;
  find_rows<true>(A, t0, n, &s_rows, false);
  // the rows that are the first of their block, in row order
  if (warp == 0) {
    bool first = false;
    if (lane < n) {
      int col;
      const int64_t p = row_place(&s_rows, t0, lane, &col);
      if (p >= 0) {
        const int4 g = s_rows.seg[lane];
        const int64_t begin = max((int64_t)g.w - g.y, (int64_t)0), b0 = p & -kPackedRows;
        first = (p == b0 || p == begin) && b0 - (begin & -kPackedRows) < A.rows;
      }
    }
    const uint32_t all = __ballot_sync(0xffffffffu, first);
    if (first) s_first[__popc(all & ((1u << lane) - 1))] = lane;
    if (lane == 0) {
      s_count = __popc(all);
      s_share = 0;
    }
  }
  __syncthreads();
  const int count = s_count;
  // every block's rows: a thread each
  static_assert(kRopeThreads == kStepRows * kPackedRows, "a thread for each row of each block");
  bool share = false;
  {
    const int f = tid / kPackedRows, row = tid % kPackedRows;
    int src = kNone, pos[kRopeAxes] = {0, 0, 0, 0};
    if (f < count) {
      const int r = s_first[f];
      const int4 g = s_rows.seg[r];
      const int64_t b0 = ((int64_t)g.w - g.y + (t0 + r - g.x)) & -kPackedRows;
      const int brow = (int)((uint32_t)b0 % (uint32_t)A.rows);
      if (row == 0) s_block.at[f] = make_int2(brow, g.z);
      src = block_row(A, g, brow + row, pos);
      share = s_rows.shared[r];
    }
    s_block.put(f, row, src, pos);
    const uint32_t fresh = __ballot_sync(0xffffffffu, src >= 0) >> (lane & kPackedRows) & 0xFFFFu;
    if (row == 0) s_block.fresh[f] = fresh != 0;
  }
  if (share) s_share = 1;
  __syncthreads();
  if (__builtin_expect(s_share != 0, 0)) share_blocks(A, s_rows, s_block, s_writers, s_first, count);
  for (int f = 0; f < count; ++f) {
    if (!s_block.fresh[f]) continue;  // (no row of the block has angles)
    const int2 at = s_block.at[f];
    Row16 x[U];
    int src[U];
#pragma unroll
    for (int u = 0; u < U; ++u) src[u] = s_block.src[f][u * RPP + ls];
    for (int i = tid; i < kPackedRows * A.r.half; i += kRopeThreads) {
      const int o = i / A.r.half, j = i - o * A.r.half;
      if (s_block.src[f][o] < 0) continue;
      int p = s_block.pos[f][o][0];
#pragma unroll
      for (int a = 1; a < kRopeAxes; ++a) p = j >= A.r.sec_end[a - 1] ? s_block.pos[f][o][a] : p;
      s_angles[o][j] = __ldg(A.r.table + (uint32_t)(p * A.r.half + j));  // below 2^31 (checked on the host)
    }
    __syncthreads();

    for (int item = warp; item < 2 * heads; item += kWarps) {
      const bool key = item < heads;
      const int h = ha + (key ? item : item - heads);
      const int64_t cell = ((int64_t)at.y * A.Hkv + h) * A.rows + at.x;
      uint8_t* codes = (key ? A.q4.kc : A.q4.vc) + cell * D;
      uint8_t* scale = (key ? A.q4.ks : A.q4.vs) + cell / kPackedRows;
      const uint32_t was = min((uint32_t)*scale, (uint32_t)kQ8Top);
      const __nv_bfloat16* rows = key ? A.k + h * A.k_hs : A.v + h * A.v_hs;
      const int64_t rs = key ? A.k_rs : A.v_rs;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (src[u] >= 0) {
          x[u].a = ldg16(rows + src[u] * rs + ld.da);
          x[u].b = ldg16(rows + src[u] * rs + ld.db);
        } else if (src[u] == kKept) {
          const uint2 a = *reinterpret_cast<const uint2*>(codes + (u * RPP + ls) * D + ld.da);
          const uint2 b = *reinterpret_cast<const uint2*>(codes + (u * RPP + ls) * D + ld.db);
          x[u].a = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
      uint32_t pairs = 0;  // largest magnitudes of the new rows, of even dims and of odd ones
      float kept = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (src[u] >= 0) {
          if (key && ld.turn) {
            Angles an;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 v = reinterpret_cast<const float4*>(s_angles[u * RPP + ls] + j0)[k];
              an.cs[2 * k] = v.x; an.sn[2 * k] = v.y;
              an.cs[2 * k + 1] = v.z; an.sn[2 * k + 1] = v.w;
            }
            turn16<IL, true>(&x[u], an);
          }
          pairs = pair_amax(pair_amax(pairs, x[u].a), x[u].b);
        } else if (src[u] == kKept) {
          kept = fmaxf(kept, fmaxf(fmaxf(q8_amax4(x[u].a.x), q8_amax4(x[u].a.y)),
                                   fmaxf(q8_amax4(x[u].a.z), q8_amax4(x[u].a.w))));
        }
      }
      uint32_t most = max(pairs & 0xFFFFu, pairs >> 16);
      if (__any_sync(0xffffffffu, most > kQ8Most)) {  // NaN, infinities, magnitudes beyond the largest scale's
        pairs = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (src[u] < 0) continue;
          x[u].a = make_uint4(q8_storable(x[u].a.x), q8_storable(x[u].a.y), q8_storable(x[u].a.z), q8_storable(x[u].a.w));
          x[u].b = make_uint4(q8_storable(x[u].b.x), q8_storable(x[u].b.y), q8_storable(x[u].b.z), q8_storable(x[u].b.w));
          pairs = pair_amax(pair_amax(pairs, x[u].a), x[u].b);
        }
        most = max(pairs & 0xFFFFu, pairs >> 16);
      }
      const float amax = __uint_as_float(
          __reduce_max_sync(0xffffffffu, max(most << 16, __float_as_uint(kept * q8_scale(was)))));
      const uint32_t byte = q8_scale_byte(amax);
      const float inv = __uint_as_float((127 + kQ8Bias - byte) << 23);
      const float ratio = q8_scale(was) * inv;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint8_t* to = codes + (u * RPP + ls) * D;
        if (src[u] >= 0) {
          *reinterpret_cast<uint2*>(to + ld.da) = q8_codes8(x[u].a, inv);
          *reinterpret_cast<uint2*>(to + ld.db) = q8_codes8(x[u].b, inv);
        } else if (src[u] == kKept && byte != was) {
          *reinterpret_cast<uint2*>(to + ld.da) = make_uint2(q8_again(x[u].a.x, ratio), q8_again(x[u].a.y, ratio));
          *reinterpret_cast<uint2*>(to + ld.db) = make_uint2(q8_again(x[u].a.z, ratio), q8_again(x[u].a.w, ratio));
        }
      }
      if (lane == 0) *scale = (uint8_t)byte;
    }
    if (f + 1 < count) __syncthreads();  // the angles are written again
  }
}

// CTAs [0, kv_ctas) code blocks, the others rotate queries.
template <int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, D == 256 ? 2 : 3) sdpa_rope_append_q8_kernel(const __grid_constant__ StepArgs A) {
  __shared__ RowTable s_rows;
  __shared__ BlockRows s_block;
  __shared__ BlockWriters s_writers;
  __shared__ int s_first[kStepRows], s_count, s_share;
  __shared__ __align__(16) float2 s_angles[kPackedRows][D / 2];
  if ((int)blockIdx.x < A.kv_ctas) {
    code_blocks<D, IL>(A, blockIdx.x, s_rows, s_block, s_writers, s_first, s_count, s_share, s_angles);
  } else {
    step_passes<D, IL, false>(A, blockIdx.x - A.kv_ctas, s_rows, s_angles,
                              [](Row16&, const LaneDims<IL>&, const Angles&, bool, int, int, int2) {});
  }
}

// Where packed row t is kept: (store row, column), or (-1, 0) when no live segment holds it or it lies before its
// sequence's beginning.  A warp's lanes look at the segments together, 32 at a time: for tables of up to kFewSegs.  With
// find_rows, which a CTA's warps do together for 16 rows, they waited at its barriers more than for anything else: 57025
// tokens of two segments 65.1 us, 61.8 so.  Tables of more take find_rows, whose 256 threads see a segment each and whose
// CTA reads the table once.  Rows of 8 heads read back, this / find_rows, us: 16 rows of each of 32 segments 4.9 / 5.1, of
// 64 6.2 / 5.9, of 256 13.3 / 8.2, of 2048 386 / 87; one row of each of 32 3.1 / 3.3, of 64 3.6 / 3.3, of 512 15.4 / 6.7.
constexpr int kFewSegs = 32;
__device__ __forceinline__ int2 find_row(const StepArgs& A, int64_t t, int lane, bool report) {
  int32_t bits = 0;
  auto load = [&](int i) -> int4 {  // entry i, empty unless it is valid
    int4 g = __ldg(reinterpret_cast<const int4*>(A.seq_info) + i);
    const int window = A.seg_mode ? __ldg(A.seg_mode + 2 * i + 1) : A.window;
    const int32_t b = segment_bits(g.x, g.y, g.z, g.w, A.T, A.rows, A.cols, window);
    bits |= b;
    if (b || g.y <= 0) g = make_int4(0, 0, 0, 0);
    return g;
  };
  int owner = -1;
  bool dead = false;
  int4 own = make_int4(0, 0, 0, 0);
  for (int base = 0; base < A.S; base += 32) {
    int4 g = make_int4(0, 0, 0, 0);
    if (base + lane < A.S) g = load(base + lane);
    const uint32_t in = __ballot_sync(0xffffffffu, t >= g.x && t < (int64_t)g.x + g.y);
    if (in == 0) continue;
    dead |= owner >= 0 || (in & (in - 1)) != 0;
    const int src = __ffs(in) - 1;
    owner = base + src;
    own = make_int4(__shfl_sync(0xffffffffu, g.x, src), __shfl_sync(0xffffffffu, g.y, src),
                    __shfl_sync(0xffffffffu, g.z, src), __shfl_sync(0xffffffffu, g.w, src));
  }
  if (report) {
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0 && bits) atomicOr(A.status_dev, bits);
  }
  // a segment that shares any row with another valid one is dropped
  for (int base = 0; owner >= 0 && !dead && base < A.S; base += 32) {
    int4 g = make_int4(0, 0, 0, 0);
    if (base + lane < A.S && base + lane != owner) g = load(base + lane);
    dead = __any_sync(0xffffffffu, max(g.x, own.x) < min(g.x + g.y, own.x + own.y));
  }
  if (dead && lane == 0 && A.status_dev) atomicOr(A.status_dev, SDPA_SEG_OVERLAP);
  const int64_t p = (int64_t)own.w - own.y + (t - own.x);
  if (owner < 0 || dead || p < 0) return make_int2(-1, 0);
  return make_int2((int)((uint32_t)p % (uint32_t)A.rows), own.z);
}

// The rows of a segment table read back from an 8-bit store as bf16 (exact), rows that no live segment holds and
// rows before a sequence's beginning as 0.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) sdpa_q8_unpack_kernel(StepArgs A) {
  constexpr int CPH = D / 16, U = 4, kWarps = kRopeThreads / 32;  // chunks of a head
  const int64_t t0 = (int64_t)blockIdx.x * A.cr;
  const int n = (int)min((int64_t)A.cr, A.T - t0);
  // A lane takes chunks of 16 dims, U at a time over the rows of its warp (warp, warp + 8).  Two lanes change
  // halves before they write, so that each write of a warp is 512 bytes in a row.
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, per = A.Hkv * CPH;
  const bool odd = lane & 1;
  static_assert(kStepRows <= 2 * kWarps, "two rows a warp");
  const bool few = A.S <= kFewSegs;
  __shared__ RowTable s_rows;
  if (!few) find_rows<false>(A, t0, n, &s_rows, blockIdx.x == 0);
  int2 cells[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = warp + k * kWarps;
    cells[k] = make_int2(-1, 0);
    if (r >= n) continue;
    if (few) {
      cells[k] = find_row(A, t0 + r, lane, k == 0 && blockIdx.x == 0 && warp == 0 && A.status_dev);
    } else {
      int col = 0;
      const int64_t p = row_place(&s_rows, t0, r, &col);
      if (p >= 0) cells[k] = make_int2((int)((uint32_t)p % (uint32_t)A.rows), col);
    }
  }
  int r = warp, x = lane;
  while (r < n) {
    uint4 kw[U], vw[U];
    uint32_t kb[U], vb[U];
    int row[U], at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row[u] = r < n && x < per ? r : -1;
      at[u] = x;
      if (row[u] >= 0) {
        const int2 from = r == warp ? cells[0] : cells[1];  // (a row that is not there reads another one's bytes)
        const int h = x / CPH, c = x % CPH;
        const int64_t cell = ((int64_t)from.y * A.Hkv + h) * A.rows + max(from.x, 0);
        kw[u] = *reinterpret_cast<const uint4*>(A.q4.kc + cell * D + 16 * c);
        vw[u] = *reinterpret_cast<const uint4*>(A.q4.vc + cell * D + 16 * c);
        kb[u] = A.q4.ks[cell / kPackedRows];
        vb[u] = A.q4.vs[cell / kPackedRows];
      }
      x += 32;
      if (x - lane >= per) {
        x = lane;
        r += kWarps;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      auto out = [&](const uint4& w, uint32_t byte, __nv_bfloat16* to) {
        const uint2 lo = make_uint2(w.x, w.y), hi = make_uint2(w.z, w.w), send = odd ? lo : hi;
        const uint2 got = make_uint2(__shfl_xor_sync(0xffffffffu, send.x, 1), __shfl_xor_sync(0xffffffffu, send.y, 1));
        if (row[u] < 0) return;
        const uint2 w0 = odd ? got : lo, w1 = odd ? hi : got;
        const bool there = (row[u] == warp ? cells[0] : cells[1]).x >= 0;
        const __nv_bfloat162 s = q8_scale_bf16(byte);
        const uint2 a = q8_words4(w0.x, s), b = q8_words4(w0.y, s), c = q8_words4(w1.x, s), d = q8_words4(w1.y, s);
        const uint4 zero = make_uint4(0, 0, 0, 0);
        stg16(to, there ? make_uint4(a.x, a.y, b.x, b.y) : zero);
        stg16(to + 16, there ? make_uint4(c.x, c.y, d.x, d.y) : zero);
      };
      const int64_t to = (t0 + max(row[u], 0)) * A.o_rs + (int64_t)(at[u] / CPH) * A.o_hs + at[u] % CPH / 2 * 32 + 8 * odd;
      out(kw[u], kb[u], A.k_out + to);
      out(vw[u], vb[u], A.v_out + to);
    }
  }
}

template <bool IL>
static const void* append_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_rope_append_q8_kernel<64, IL>;
    case 128: return (const void*)sdpa_rope_append_q8_kernel<128, IL>;
    default: return (const void*)sdpa_rope_append_q8_kernel<256, IL>;
  }
}
const void* rope_append_q8_kernel_ptr(int D, bool il) { return il ? append_ptr<true>(D) : append_ptr<false>(D); }
const void* q8_unpack_kernel_ptr(int D) {
  switch (D) {
    case 64: return (const void*)sdpa_q8_unpack_kernel<64>;
    case 128: return (const void*)sdpa_q8_unpack_kernel<128>;
    default: return (const void*)sdpa_q8_unpack_kernel<256>;
  }
}

}  // namespace sdpa
