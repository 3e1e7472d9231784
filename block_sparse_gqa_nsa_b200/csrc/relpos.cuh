// Shared pieces of the attention with a learned relative position bias by buckets.  Which file has which
// kernels: relpos.cu forward of few and of some tens of queries a segment, joins; relpos_short.cu forward and
// dq of many short segments; relpos_tc.cu forward of long ones on tcgen05; relpos_bwd.cu the backward's
// mathematics, its kernels up to middle lengths, joins; relpos_bwd_tc.cu the backward of long segments.
//
// Segment s holds the queries off_q[s] .. off_q[s+1]-1 and the keys off_k[s] .. off_k[s+1]-1; every
// query attends every key of its segment.  With D = max_distance, per axis a of the positions
//   delta_a = clamp(pos_k[j][a] - pos_q[i][a], -D, D)
//   t_ijh   = scale q_ih . k_j,g(h) + sum_a table[a][bucket_of[delta_a + D]][h]
//   lse_ih  = log sum_j exp(t_ijh),  o_ih = sum_j exp(t_ijh - lse_ih) v_j,g(h)
// and a row without keys (or with every t at -inf) has o = 0 and lse = -inf.
#pragma once

#include <climits>

#include "dependent.cuh"
#include "tc_ptx.cuh"

namespace lsrm {
namespace rp {

constexpr int kPosLimit = 1 << 29;  // positions lie in [-2^29, 2^29], so differences stay in 32 bits
constexpr int kMaxBuckets = 64;
constexpr int kMaxDistance = 1023;
constexpr int kMaxAxes = 3;
using tc::fadd2_acc;
using tc::ffma2;
using tc::fmax3;
using tc::fmul2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Arithmetic without side effects, so not `asm volatile`: volatile statements keep their order, and a
// kernel that interleaves exponentials, packing and products would wait out each one's latency in turn.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// r = (a0, a1) * (b, b) + (c0, c1)
__device__ __forceinline__ void ffma2v(float& r0, float& r1, float a0, float a1, float b, float c0, float c1) {
  uint64_t ra, rb, rc, rd;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(ra) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %1};\n" : "=l"(rb) : "f"(b));
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(rc) : "f"(c0), "f"(c1));
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;\n" : "=l"(rd) : "l"(ra), "l"(rb), "l"(rc));
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r0), "=f"(r1) : "l"(rd));
}
// In a rarely taken branch: keeps it a branch, where the compiler would rather do both sides and select
__device__ __forceinline__ void keep_branch() { asm volatile("" ::: "memory"); }

// A bias folds into the exponent's multiply-add, in whatever order is cheapest, only while scores are small
// beside fp32's spacing.  Tables with larger entries than kSmallBias (a mask of the type's lowest value), and in the
// backward rows whose |LSE| reaches kFoldLimit (spacing 2^-10), take the exact path: t = ((s scale) + b_0) + b_1 + b_2
// in the formula's own order, so that both backward passes have the same t bit for bit, whatever their tiles have in
// common, and the row's reference subtracted from it before anything else.
//
// LSE itself loses the logarithm of a row's sum beside a large score.  So the backward's weights are
// exp(t - lse) / sum_j exp(t - lse): the dq pass adds the sums up beside its products and hands their log2 (corr) to
// the key pass.
constexpr float kFoldLimit = 1e4f;
constexpr float kSmallBias = 64.0f;  // per axis: three axes in log2 units keep a spacing of 2^-15

struct Params {
  const int32_t* off_q;
  const int32_t* off_k;
  const int32_t* pos_q;
  const int32_t* pos_k;
  const int32_t* bucket_of;
  const uint16_t* table;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;
  const uint16_t* o_in;  // backward: the forward's out
  const float* lse_in;
  const uint16_t* dout;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  uint16_t* dtable;
  float* delta;  // backward: Delta per (query, head)
  float* tab_part;  // backward: table gradient per (key tile, part of its queries, head)
  float* kv_part;   // backward: dK / dV per split
  float* corr;      // backward: log2 of what exp(t - lse) sums to per (query, head)
  float* lse2;      // backward: lse in log2 units with corr, +inf for a row without keys
  float* o_part;    // forward: output per key split, and its softmax reference and sum
  float2* ml_part;
  uint32_t* status;
  int Nq, Nk, S, Hq, Hkv, G, NB, maxd;
  int splits;
  float scale;
};

// ---- segments ----
// Bounds of segment s, clipped to [0, n] and to each other so that a wrong table cannot lead out of
// the tensors (it raises LSRM_ERR_BOUNDS).
__device__ __forceinline__ void seg_bounds(const int32_t* off, int s, int n, int& lo, int& hi, uint32_t* status) {
  const int a = off[s], b = off[s + 1];
  lo = min(max(a, 0), n);
  hi = min(max(b, lo), n);
  if (lo != a || hi != b) raise_status(status, LSRM_ERR_BOUNDS);
}

// Tiles of R rows cut from the segments, numbered without a prefix sum: segment s starts at tile
// off[s] / R + s, which leaves it at least ceil(len / R) numbers, and all numbers are below
// n / R + segments.  The segment of a number is the last one that starts at or before it, found by a
// search with 32 probes a round (the warp's lanes), so 1000 segments take two dependent reads; whole
// warps only.  Numbers behind a segment's last tile are empty.
__device__ __forceinline__ int seg_of_tile(const int32_t* off, int S, int n, int R, int tile, int& first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = S;  // the segment lies in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) >> 5, mid = lo + lane * step;
    const bool before = lane * step < len && min(max(off[mid], 0), n) / R + mid <= tile;
    const int k = max(31 - __clz(__ballot_sync(0xffffffffu, before)), 0);  // the last probe at or before it
    len = min(step, lo + len - (lo + k * step));
    lo += k * step;
  }
  first = min(max(off[lo], 0), n) / R + lo;
  return lo;
}

// ---- the bias of one head by clamped distance, in shared memory ----
__device__ __forceinline__ int checked_bucket(const Params& p, int i) {
  const int b = p.bucket_of[i];
  if (b < 0 || b >= p.NB) {
    raise_status(p.status, LSRM_ERR_BOUNDS);
    return -1;
  }
  return b;
}

// clamp(x + y, 0, top) in one instruction; any wrap-around stays in the table
__device__ __forceinline__ int clamp_index(int x, int y, int top) { return __viaddmin_s32_relu(x, y, top); }

// ---- tiles in shared memory ----
// A score tile of 32 columns: the accumulator layout gives the lane with tq = lane % 4 the columns
// 2 tq, 2 tq + 1 of each of the four groups of 8.  Which stored row a column stands for is free (the
// softmax and the sums do not care), so column 2 tq + e of group n is stored row 8 tq + 2 n + e: a lane
// then holds 8 consecutive tokens, whose positions often are the same on an axis (one look-up for all
// of them) and load as vectors.
//
// Rows of D bf16 lie in 16-byte pieces, swizzled so that the eight rows of one 8x8 matrix (0, 1, 8, 9,
// 16, .. behind 2 n) fall into different banks.
constexpr int kCols = 32, kGroups = 4, kLaneCols = 8;
template <int D>
__device__ __forceinline__ int piece(int row, int c) {
  return D == 32 ? row * 4 + (c ^ ((row >> 3) & 3)) : row * 8 + (c ^ ((row & 1) | ((row >> 2) & 6)));
}

// rows [r0, r0 + n_valid) of a [tokens][heads][D] tensor, head h; rows past n_valid are filled with zeros
template <int D, int ROWS, int NT>
__device__ __forceinline__ void load_tile(uint4* dst, const uint16_t* src, int r0, int n_valid, int heads, int h,
                                          int tid) {
  constexpr int kPieces = D / 8;
  static_assert(NT % kPieces == 0 && ROWS * kPieces % NT == 0, "a thread keeps its column, all have as many rows");
  const int c = tid % kPieces, step = heads * D;
  const uint16_t* from = src + ((size_t)r0 * heads + h) * D + c * 8;
#pragma unroll
  for (int i = 0; i < ROWS * kPieces / NT; ++i) {
    const int r = tid / kPieces + i * (NT / kPieces);
    const bool ok = r < n_valid;
    cp_async16(dst + piece<D>(r, c), from + (ok ? r * step : 0), ok);  // (65535 heads x 64 x 64 rows fit 32 bits)
  }
}
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem, bool pred) {
  const int n = pred ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(smem)), "l"(gmem), "r"(n));
}

// B operand for X Y^T: column group n (8 columns) by all of D (k): b[2 * ks], b[2 * ks + 1] per k step
template <int D>
__device__ __forceinline__ void load_b_rows(uint32_t* b, const uint4* tile, int row0, int n, int lane) {
  const int row = row0 + ((lane & 7) >> 1) * kLaneCols + 2 * n + (lane & 1);
#pragma unroll
  for (int c = 0; c < D / 8; c += 4) {
    const uint32_t a = smem_u32(tile + piece<D>(row, c + (lane >> 3)));
    ldmatrix_x4(b[c], b[c + 1], b[c + 2], b[c + 3], a);
  }
}
// B operand for P Y: column groups 2 j and 2 j + 1 (16 rows of Y, k) by columns [8 c, 8 c + 16) of Y
template <int D>
__device__ __forceinline__ void load_b_cols(uint32_t* b, const uint4* tile, int row0, int j, int c, int lane) {
  const int row = row0 + ((lane & 7) >> 1) * kLaneCols + 2 * (2 * j + ((lane >> 3) & 1)) + (lane & 1);
  ldmatrix_x4_trans(b[0], b[1], b[2], b[3], smem_u32(tile + piece<D>(row, c + (lane >> 4))));
}
// A operand straight from global memory: rows g and g + 8 of a 16-row tile; row pointers may be null
template <int D>
__device__ __forceinline__ void load_a_rows(uint32_t (*a)[4], const uint16_t* r0, const uint16_t* r1, int lane) {
  const int t = lane & 3;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const int c = ks * 16 + 2 * t;
    a[ks][0] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c) : 0u;
    a[ks][1] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c) : 0u;
    a[ks][2] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c + 8) : 0u;
    a[ks][3] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c + 8) : 0u;
  }
}

__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// ---- what a tile's distances have in common ----
// Per axis, for a warp's tile of 32 columns whose column positions are xs[col * NA]:
//   kOne   every (row, column) pair has one clamped distance (all pairs at or past +-maxd, or single
//          positions): one look-up for the tile;
//   kLane  each lane's columns have one position: one look-up per row;
//   kFour  aligned runs of four columns have one position: one look-up per row and run;
//   kTurn  the same four positions in every run: four look-ups per row;
//   kEach  a look-up per pair (following arbitrary runs with a branch per column measured 10-20% slower
//          on every training case: the branches cost more than the look-ups they save).
// Lattice orders (bricks, patches, frames) make the slow axes kLane or kFour, bricks of four the fast one
// kTurn; distances past max_distance make kOne.  The tests cost about 20 instructions a tile and axis.
enum : int { kOne = 0, kLane = 1, kFour = 2, kTurn = 3, kEach = 4 };

template <int NA>
__device__ __forceinline__ int axis_mode(const int* xs, int row_lo, int row_hi, bool rows_are_keys, int maxd, int lane,
                                         int& one, uint32_t* status) {
  const int x = xs[lane * NA];
  const int lo = __reduce_min_sync(0xffffffffu, x), hi = __reduce_max_sync(0xffffffffu, x);
  if (lo < -kPosLimit || hi > kPosLimit) raise_status(status, LSRM_ERR_BOUNDS);
  const int a = clamp_index(rows_are_keys ? row_lo - hi : lo - row_hi, maxd, 2 * maxd);
  const int b = clamp_index(rows_are_keys ? row_hi - lo : hi - row_lo, maxd, 2 * maxd);
  one = a;
  if (a == b) return kOne;
  const uint32_t same = __ballot_sync(0xffffffffu, x == __shfl_down_sync(0xffffffffu, x, 1));
  if ((same & 0x7f7f7f7fu) == 0x7f7f7f7fu) return kLane;
  if ((same & 0x77777777u) == 0x77777777u) return kFour;
  const uint32_t turn = __ballot_sync(0xffffffffu, x == __shfl_down_sync(0xffffffffu, x, 4));
  return (turn & 0x0f0f0f0fu) == 0x0f0f0f0fu ? kTurn : kEach;
}

// The bias table of one head in shared memory, and whether it may fold: in log2 units (true) when every
// entry is small or -inf, so that bias, reference and units become one multiply-add of the exponent; in
// natural units (false) otherwise.  A CTA-wide call with barriers on both sides of the table.
template <int NA, int NT>
__device__ __forceinline__ bool fill_units(const Params& p, float* lut, int h, int tid) {
  const int n = 2 * p.maxd + 1;
  bool small = true;
  for (int i = tid; i < n; i += NT) {
    const int b = checked_bucket(p, i);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const float x = b < 0 ? 0.0f : bf16_to_f32(p.table[((size_t)a * p.NB + b) * p.Hq + h]);
      small = small && (fabsf(x) <= kSmallBias || x == -INFINITY);
      lut[a * n + i] = x;
    }
  }
  const bool fold = __syncthreads_and(small);
  if (fold) {  // every thread scales the entries that it wrote
    for (int i = tid; i < n; i += NT)
#pragma unroll
      for (int a = 0; a < NA; ++a) lut[a * n + i] *= kLog2e;
  }
  __syncthreads();
  return fold;
}

// The bias of a lane's MT x 2 rows by 8 columns, in the table's units.  What is constant per row goes
// to base; when that is all, returns true and leaves the scores raw.  Otherwise the scores become
// s * mul + bias; `exact`: in the formula's own order, whatever the modes, and base is 0.  SIGN: column positions
// count up (+1, columns are keys: rowc = maxd - pos_q) or down (-1, columns are queries: rowc = maxd + pos_k).
template <int NA, int MT, int SIGN>
__device__ __forceinline__ bool add_bias(float (&s)[MT][kGroups][4], float (&base)[MT][2], const int (&mode)[NA],
                                         const int (&one)[NA], const int* xs, const float* lut, int top,
                                         const int (&rowc)[MT][2][NA], float mul, bool exact, int tq) {
  const int* mine = xs + tq * kLaneCols * NA;
  int worst = kOne;
  float ub = 0.0f;
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    worst = max(worst, mode[a]);
    if (mode[a] == kOne && !exact) ub += lut[a * (top + 1) + one[a]];
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) base[mt][0] = base[mt][1] = ub;
  if (!exact) {
    if (worst == kOne) return true;
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      if (mode[a] != kLane) continue;
      const int x = SIGN * mine[a];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) base[mt][i] += lut[a * (top + 1) + clamp_index(x, rowc[mt][i][a], top)];
    }
    if (worst <= kLane) return true;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < kGroups; ++n)
        ffma2(s[mt][n][2 * i], s[mt][n][2 * i + 1], s[mt][n][2 * i], s[mt][n][2 * i + 1], mul, base[mt][i]);
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    const float* la = lut + a * (top + 1);
    if (mode[a] == kFour) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int x = SIGN * mine[4 * r * NA + a];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float b = la[clamp_index(x, rowc[mt][i][a], top)];
            s[mt][2 * r][2 * i] += b, s[mt][2 * r][2 * i + 1] += b;
            s[mt][2 * r + 1][2 * i] += b, s[mt][2 * r + 1][2 * i + 1] += b;
          }
      }
    } else if (mode[a] == kTurn) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int x0 = SIGN * mine[2 * n * NA + a], x1 = SIGN * mine[(2 * n + 1) * NA + a];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float b0 = la[clamp_index(x0, rowc[mt][i][a], top)], b1 = la[clamp_index(x1, rowc[mt][i][a], top)];
            s[mt][n][2 * i] += b0, s[mt][n][2 * i + 1] += b1;
            s[mt][n + 2][2 * i] += b0, s[mt][n + 2][2 * i + 1] += b1;
          }
      }
    } else if (mode[a] == kEach) {
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        const int x0 = SIGN * mine[2 * n * NA + a], x1 = SIGN * mine[(2 * n + 1) * NA + a];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // single adds: a pair of look-ups would first have to be moved into a pair of registers
            s[mt][n][2 * i] += la[clamp_index(x0, rowc[mt][i][a], top)];
            s[mt][n][2 * i + 1] += la[clamp_index(x1, rowc[mt][i][a], top)];
          }
      }
    } else if (exact) {  // (otherwise in base)
      keep_branch();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float b = la[mode[a] == kOne ? one[a] : clamp_index(SIGN * mine[a], rowc[mt][i][a], top)];
#pragma unroll
          for (int n = 0; n < kGroups; ++n) s[mt][n][2 * i] += b, s[mt][n][2 * i + 1] += b;
        }
    }
  }
  return false;
}

// ---- backward ----
// the LSE that the exponents take: a row without keys has P = 0
__device__ __forceinline__ float row_lse(float lse) { return lse == -INFINITY ? INFINITY : lse; }
// the row constant of the scores' units, subtracted from them in the exact path.  (Rounded by itself: both passes
// need the same number.)
__device__ __forceinline__ float row_const(float lse, bool small) { return small ? __fmul_rn(lse, kLog2e) : lse; }
__device__ __forceinline__ bool is_huge(float x) { return fabsf(x) >= kFoldLimit && x != INFINITY; }
// 1 / l of a row's weights exp(t - lse), 0 for a row without keys.  A sum that left fp32's range means that lse is not
// the forward's, or that scores are so large (past 2^27, where the two passes' own roundings of one score, a few times
// 2^-24 of it, differ by tens) that it says nothing about them.
__device__ __forceinline__ float row_inverse(float l, float row, uint32_t* status) {
  if ((l == 0.0f || l == INFINITY) && fabsf(row) < INFINITY) raise_status(status, LSRM_ERR_BOUNDS);
  return l == 0.0f ? 0.0f : 1.0f / l;
}
__device__ __forceinline__ float row_corr(float l) { return l == 0.0f ? 0.0f : log2f(l); }
__device__ __forceinline__ float row_lse2(float row, bool small, float corr) {
  return small ? row + corr : fmaf(row, kLog2e, corr);
}

// Two sums into a column of the table's gradient (byte offsets of the buckets' entries) with both reads ahead
// of both writes: one latency for two, and right when the buckets are the same.
__device__ __forceinline__ void add_two(char* col, int b0, float v0, int b1, float v1) {
  float *p0 = reinterpret_cast<float*>(col + b0), *p1 = reinterpret_cast<float*>(col + b1);
  const float s0 = *p0 + v0, x1 = *p1;
  *p0 = s0;
  *p1 = (b0 == b1 ? s0 : x1) + v1;
}

// A head's table gradient from its columns hist[axis][NB and one for ids out of range][COLS]: the sum of each
// bucket's columns to out[bins], and the columns back to 0.  One to four threads a bucket walk its columns,
// each from another bank, so that a warp's reads meet no conflict and hardly a shuffle is left (dk/dv of 256
// ragged blocks of up to 64 tokens, 32 heads: 138 us; a warp a bucket, joined by shuffles, 155).
// Called by THREADS threads between barriers.
template <int COLS, int THREADS>
__device__ __forceinline__ void flush_sums(float* hist, int bins, int nb, int tid, float* out) {
  const int shift = 4 * bins <= THREADS ? 2 : 2 * bins <= THREADS ? 1 : 0, width = COLS >> shift;
  for (int i0 = 0; i0 < bins << shift; i0 += THREADS) {
    const int i = i0 + tid, b = i >> shift;
    float x = 0.0f;
    if (b < bins) {
      // past each axis' entry for ids out of range
      float* of = hist + (b + (b >= nb) + (b >= 2 * nb)) * COLS + (i & ((1 << shift) - 1)) * width;
#pragma unroll 8
      for (int k = 0; k < width; ++k) {
        float* at = of + ((i + k) & (width - 1));
        x += *at;
        *at = 0.0f;
      }
    }
    if (shift > 0) x += __shfl_xor_sync(0xffffffffu, x, 1);
    if (shift > 1) x += __shfl_xor_sync(0xffffffffu, x, 2);
    if (b < bins && (i & ((1 << shift) - 1)) == 0) out[b] = x;
  }
}

// the (head, query chunk) range of a split: whole heads, or an even part of one head's chunks
__device__ __forceinline__ void split_range(const Params& p, int split, int chunks, int& h0, int& h1, int& c0, int& c1,
                                            int& part) {
  if (p.splits <= p.G) {
    const int n = p.G / p.splits;
    h0 = split * n, h1 = h0 + n, c0 = 0, c1 = chunks, part = 0;
  } else {
    const int f = p.splits / p.G, n = (chunks + f - 1) / f;
    h0 = split / f, h1 = h0 + 1, part = split % f;
    c0 = min(part * n, chunks), c1 = min(c0 + n, chunks);
  }
}

// ---- launch plans and the workspace (host) ----
// A kernel's limit of dynamic shared memory belongs to the kernel, so it is always the same, whatever this call
// needs: a second thread with a smaller table cannot lower it between a call's setting and its launch.
constexpr int kSmemMost = 227 * 1024;
template <typename K>
inline bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 48 * 1024 ||
         (bytes <= (size_t)kSmemMost &&
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) == cudaSuccess);
}

constexpr int kSms = 148;
constexpr int kShHeads = 16;                 // heads a CTA of the short segments' kernels takes, at most
constexpr size_t kShTables = 64 * 1024;      // bytes of their bias tables, at most
inline size_t short_tables(const lsrm_relpos_desc& d) {
  const size_t g = (size_t)(d.n_q_heads / d.n_kv_heads);
  return (g < kShHeads ? g : kShHeads) * d.n_axes * (2 * (size_t)d.max_distance + 1) * 4;
}
inline long long short_ctas(const lsrm_relpos_desc& d) {
  const long long g = d.n_q_heads / d.n_kv_heads, gh = g < kShHeads ? g : kShHeads;
  return (d.n_q_tokens / 64 + d.n_segs) * d.n_kv_heads * ((g + gh - 1) / gh);
}

struct FwdPlan {
  int rows;  // queries a CTA: 256 (tensor-memory kernel), 128, 64, 0 for the kernel of few rows, -1 for short segments
  int splits;
  long long ctas;
};
struct BwdPlan {
  int tc;       // the tensor-memory kernels of 128 rows a CTA: CTAs of the key pass an SM holds, or 0
  bool shrt;    // short segments' dq kernel
  int splits;   // of the key pass over heads and query chunks: a divisor of G, or a multiple of it
  int g;
  long long dq_tiles, kv_tiles, short_ctas;
  int parts() const { return splits > g ? splits / g : 1; }  // table sums per (key tile, head)
};
// The backward's tensor-memory kernels past this many keys, from where a 128-row key tile is as full as two of 64:
// backward of eight segments, three axes and 32 heads of 32, 512 queries against 64 keys 154 us (64-row kernels 117), 110
// keys on one axis 93 (100); 16 heads of 64, 300 queries against 80 keys 90 (104), 160 keys 78 (136).
constexpr int kTcKeys = 64;

int bwd_tc_ctas(int D, int NA, int maxd, int nb);  // CTAs of rp_dkv_tc_kernel an SM holds, 0: too large

// The kernel of few rows: 24 rows of 32 heads of 32 against 16 x 512 keys 29 us, 64-row tiles 41; 48 rows
// 52 us against 43 (three axes; on one axis 32 rows 21 against 27, with 16 heads of their own 48 rows 19 against 25)
constexpr int kFewRows = 24;

// Short segments' kernels: while a segment is a tile of queries or so, enough of them fill the GPU, the tables of a
// group's heads fit, and the group has heads for the eight warps.  Segments of 64 tokens, 32 heads of 32 on 2 KV heads,
// forward and backward: 64 of them 54 and 154 us, by the kernels of longer segments 37 and 129; 128 of them 56 and 206
// against 66 and 214.  Four heads a group, 256 of 40 tokens: 27 and 111 against 29 and 109; heads of their own, 128 of 64
// tokens: 55 and 144 against 30 and 114.
constexpr int kShGroup = 4;
inline bool short_kernels(const lsrm_relpos_desc& d) {
  if (d.n_q_heads / d.n_kv_heads < kShGroup) return false;
  const long long S = d.n_segs, mean_q = (d.n_q_tokens + S - 1) / S, mean_k = (d.n_k_tokens + S - 1) / S;
  return mean_q <= 64 && mean_k <= 64 && short_tables(d) <= kShTables && 3 * S * d.n_kv_heads >= 4 * kSms;
}

inline FwdPlan fwd_plan(const lsrm_relpos_desc& d) {
  FwdPlan f{};
  const long long S = d.n_segs, Nq = d.n_q_tokens, G = d.n_q_heads / d.n_kv_heads;
  const long long mean_q = (Nq + S - 1) / S, mean_k = (d.n_k_tokens + S - 1) / S;
  long long busy, chunks;  // CTAs with work, about; key chunks of an average segment
  long long want, most;    // CTAs that splits of the keys shall make, and splits at most
  if (mean_q <= kFewRows) {
    const long long gh = G < 16 ? G : 16, t = 16 / gh, hgroups = (G + gh - 1) / gh;
    f.rows = 0;
    f.ctas = (Nq / t + S) * d.n_kv_heads * hgroups;
    busy = ((mean_q + t - 1) / t) * (Nq < S ? Nq : S) * d.n_kv_heads * hgroups;
    chunks = (mean_k + 127) / 128;  // four warps of 32 keys
    // four CTAs an SM, no part below 512 keys: one token of 32 heads against 64 ragged pasts 28.9 us (two CTAs
    // 37.0), against 8 x 8192 keys 22.7 us (no part below 256 keys 31.3)
    want = 4 * kSms, most = chunks / 4;
  } else if (short_kernels(d)) {
    f.rows = -1;
    f.splits = 1;
    f.ctas = short_ctas(d);
    return f;
  } else {
    f.rows = mean_q <= 64 ? 64 : mean_q <= 96 && d.head_dim == 32 ? 128 : 256;
    f.ctas = (Nq / f.rows + S) * d.n_q_heads;
    busy = ((mean_q + f.rows - 1) / f.rows) * S * d.n_q_heads;
    chunks = (mean_k + 63) / 64;
    // As many as an SM holds.  Of the 256-row kernel two: 512 queries against 4096 keys, 32 heads of 32, 76 us (one
    // 110, four 91), 1024 tokens 33 (33, 39); of 64 and 128 rows three: 16 segments of up to 64 queries against 512
    // keys 41 to 43 us (eight 47 to 52).
    want = (f.rows == 256 ? 2 : 3) * kSms, most = chunks / 4;
  }
  long long sp = busy > 0 && busy < want ? want / busy : 1;
  if (sp > most) sp = most;
  if (sp > 64) sp = 64;
  if (sp < 1) sp = 1;
  f.splits = (int)sp;
  f.ctas *= sp;
  return f;
}

// The key pass' splits: whole heads of a group (divisors of G) or parts of one head's query chunks.
inline BwdPlan bwd_plan(const lsrm_relpos_desc& d) {
  BwdPlan b{};
  const long long S = d.n_segs, G = d.n_q_heads / d.n_kv_heads;
  const long long mean_q = (d.n_q_tokens + S - 1) / S, mean_k = (d.n_k_tokens + S - 1) / S;
  b.g = (int)G;
  // From what length 128-row tiles fill up enough, whole backward of eight segments: 16 heads of 64, two axes, 128
  // tokens 69 us (64-row kernels 56), 192 tokens 56 (100); 32 heads of 32, three axes, 320 tokens 205 us (194), 384
  // tokens 232 (289).
  b.tc = mean_k > kTcKeys && mean_q > (d.head_dim == 64 ? 128 : 320)
             ? bwd_tc_ctas(d.head_dim, d.n_axes, d.max_distance, d.n_buckets)
             : 0;
  const int rows = b.tc ? 128 : 64;
  b.shrt = short_kernels(d);
  b.short_ctas = short_ctas(d);
  b.dq_tiles = d.n_q_tokens / rows + S;
  b.kv_tiles = d.n_k_tokens / rows + S;
  const long long busy = ((mean_k + rows - 1) / rows) * S * d.n_kv_heads;
  const long long qchunks = (mean_q + 63) / 64;
  long long sp = 1;
  if (b.tc) {
    // The time in chunks of work: CTAs that an SM runs one after the other (whole ones while there are few,
    // later they even out) times a CTA's chunks and 2.5 for its beginning and end.  More splits only where they
    // win 2%, as their sums have to be joined.  Whole backward, 32 heads of 32 on three axes: 1024 tokens 16 splits 177
    // us, 8 splits 254, 32 splits 188; 8 x 384 tokens 232 us, 16 splits 238, 4 splits 259; 4096 tokens 16 splits 2292 us,
    // 8 splits 2359 (32 splits would take 2197).
    double best = 0.0;
    for (long long c = 1; c <= 64 * G && c <= G * (qchunks > 1 ? qchunks : 1); c = c < G ? c + 1 : c + G) {
      if (c < G && G % c) continue;
      const double waves = (double)(busy * c) / (b.tc * kSms);
      const double steps = c <= G ? (double)(G / c * qchunks) : (double)((qchunks + c / G - 1) / (c / G));
      const double cost = (waves <= 1 ? 1 : waves <= 2 ? 2 : waves + 0.3) * (steps + 2.5);
      if (c == 1 || cost < 0.98 * best) best = cost, sp = c;
    }
  } else {
    // 8 CTAs an SM (key pass of 256 ragged blocks of up to 64 tokens 134 us; 4 an SM 142)
    sp = busy > 0 ? (8 * kSms + busy - 1) / busy : 1;
    if (sp > 64 * G) sp = 64 * G;
    if (sp < G) {
      while (G % sp) ++sp;  // whole heads, evenly
    } else {
      sp = sp / G;          // chunks of one head
      if (sp > qchunks) sp = qchunks;
      sp = (sp < 1 ? 1 : sp) * G;
    }
  }
  b.splits = (int)sp;
  return b;
}

struct Ws {
  size_t status, o_part, ml_part, delta, corr, lse2, tab_part, kv_part, total;
};
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
// the forward's and the backward's scratch share the space behind the status word
inline Ws ws_layout(const lsrm_relpos_desc& d) {
  Ws w{};
  const size_t rows = (size_t)d.n_q_tokens * d.n_q_heads, D = d.head_dim;
  const FwdPlan f = fwd_plan(d);
  const BwdPlan b = bwd_plan(d);
  size_t o = up256(16);
  w.o_part = o;
  const size_t parts = f.splits > 1 ? (size_t)f.splits * rows : 0;
  w.ml_part = up256(w.o_part + parts * D * 4);
  const size_t fwd = up256(w.ml_part + parts * 8);
  w.delta = o;
  w.corr = up256(w.delta + rows * 4);
  w.lse2 = up256(w.corr + rows * 4);
  w.tab_part = up256(w.lse2 + rows * 4);
  w.kv_part = up256(w.tab_part + (size_t)b.kv_tiles * b.parts() * d.n_q_heads * d.n_axes * d.n_buckets * 4);
  const size_t kv = b.splits > 1 ? (size_t)b.splits * 2 * d.n_k_tokens * d.n_kv_heads * D : 0;
  const size_t bwd = up256(w.kv_part + kv * 4);
  w.total = fwd > bwd ? fwd : bwd;
  return w;
}

}  // namespace rp
}  // namespace lsrm
