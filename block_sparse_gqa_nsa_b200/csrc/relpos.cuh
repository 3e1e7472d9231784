// Shared pieces of the attention with a learned relative position bias by buckets
// (relpos.cu: forward, relpos_bwd.cu: backward).
//
// Segment s holds the queries off_q[s] .. off_q[s+1]-1 and the keys off_k[s] .. off_k[s+1]-1; every
// query attends every key of its segment.  With D = max_distance, per axis a of the positions
//   delta_a = clamp(pos_k[j][a] - pos_q[i][a], -D, D)
//   t_ijh   = scale q_ih . k_j,g(h) + sum_a table[a][bucket_of[delta_a + D]][h]
//   lse_ih  = log sum_j exp(t_ijh),  o_ih = sum_j exp(t_ijh - lse_ih) v_j,g(h)
// and a row without keys (or with every t at -inf) has o = 0 and lse = -inf.
#pragma once

#include <climits>

#include "lsrm_common.cuh"

namespace lsrm {
namespace rp {

constexpr int kPosLimit = 1 << 29;  // positions lie in [-2^29, 2^29], so differences stay in 32 bits
constexpr int kMaxBuckets = 64;
constexpr int kMaxDistance = 1023;
constexpr int kMaxAxes = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  float* tab_part;  // backward: table gradient per (query tile, head)
  float* kv_part;   // backward: dK / dV per split
  float* corr;      // backward: log2 of what exp(t - lse) sums to per (query, head), 0 for all but huge |lse|
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
// n / R + segments.  The segment of a number is found by bisection; numbers behind a segment's last
// tile are empty.
__device__ __forceinline__ int seg_of_tile(const int32_t* off, int S, int n, int R, int tile, int& first) {
  int lo = 0, hi = S - 1;  // the last segment that starts at or before the tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (min(max(off[mid], 0), n) / R + mid <= tile)
      lo = mid;
    else
      hi = mid - 1;
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
template <int NA>
__device__ __forceinline__ void fill_lut(const Params& p, float* lut, int h, int tid, int nthreads) {
  const int n = 2 * p.maxd + 1;
  for (int i = tid; i < n; i += nthreads) {
    const int b = checked_bucket(p, i);
#pragma unroll
    for (int a = 0; a < NA; ++a)
      lut[a * n + i] = b < 0 ? 0.0f : bf16_to_f32(p.table[((size_t)a * p.NB + b) * p.Hq + h]);
  }
}

// clamp(x + y, 0, top) in one instruction; any wrap-around stays in the table
__device__ __forceinline__ int clamp_index(int x, int y, int top) { return __viaddmin_s32_relu(x, y, top); }

// ---- tiles in shared memory ----
// rows of D bf16 in 16-byte pieces, swizzled so that the eight rows of an 8x8 matrix lie in
// different banks (64-byte rows: two rows fill the 32 banks; 128-byte rows: one)
template <int D>
__device__ __forceinline__ int piece(int row, int c) {
  return D == 32 ? row * 4 + (c ^ ((row >> 1) & 3)) : row * 8 + (c ^ (row & 7));
}

// rows [r0, r0 + n) of a [tokens][heads][D] tensor, head h; rows past n_valid are filled with zeros
template <int D, int ROWS, int NT>
__device__ __forceinline__ void load_tile(uint4* dst, const uint16_t* src, int r0, int n_valid, int heads, int h,
                                          int tid) {
  constexpr int kPieces = D / 8;
#pragma unroll
  for (int i = tid; i < ROWS * kPieces; i += NT) {
    const int r = i / kPieces, c = i % kPieces;
    const bool ok = r < n_valid;
    cp_async16(dst + piece<D>(r, c), src + ((size_t)(r0 + (ok ? r : 0)) * heads + h) * D + c * 8, ok);
  }
}
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem, bool pred) {
  const int n = pred ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(smem)), "l"(gmem), "r"(n));
}

// B operand for X Y^T: the 8 rows at `row` (n) by all of D (k): b[2 * ks], b[2 * ks + 1] per k step
template <int D>
__device__ __forceinline__ void load_b_rows(uint32_t* b, const uint4* tile, int row, int lane) {
#pragma unroll
  for (int c = 0; c < D / 8; c += 4) {
    const uint32_t a = smem_u32(tile + piece<D>(row + (lane & 7), c + (lane >> 3)));
    ldmatrix_x4(b[c], b[c + 1], b[c + 2], b[c + 3], a);
  }
}
// B operand for P Y: the 16 rows at `row` (k) by columns [8 c, 8 c + 16) (two n tiles)
template <int D>
__device__ __forceinline__ void load_b_cols(uint32_t* b, const uint4* tile, int row, int c, int lane) {
  const uint32_t a = smem_u32(tile + piece<D>(row + (lane & 15), c + (lane >> 4)));
  ldmatrix_x4_trans(b[0], b[1], b[2], b[3], a);
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

// ---- distances that are the same for a whole tile ----
// Index into the bias table when every (row, column) pair of the tile has the same clamped distance
// on this axis, else -1: all pairs at or past +-maxd, or both position ranges single values.
__device__ __forceinline__ int uniform_index(int k_lo, int k_hi, int q_lo, int q_hi, int maxd) {
  const int lo = clamp_index(k_lo - q_hi, maxd, 2 * maxd), hi = clamp_index(k_hi - q_lo, maxd, 2 * maxd);
  return lo == hi ? lo : -1;
}


// A bias common to a tile folds into the exponent's multiply-add only while it is small beside
// fp32's spacing: past this a score is added to it first, so that scores the addition swallows (a
// mask of the type's lowest value) count as equal, as they do in the formula's own order.
// The same size of LSE is where its own fp32 spacing (2^-10 at 1e4) begins to lose the logarithm of
// the row's sum, so the backward normalises such rows anew.
constexpr float kFoldLimit = 1e4f;

// ---- launch plans and the workspace (host) ----
constexpr int kSms = 148;

struct FwdPlan {
  int rows;  // queries a CTA: 128, 64, or 0 for the kernel of few rows
  int splits;
  long long ctas;
};
struct BwdPlan {
  int splits;  // of the (head, query chunk) loop of the key pass
  long long dq_tiles, kv_tiles;
};
constexpr int kBwdRows = 64;

inline FwdPlan fwd_plan(const lsrm_relpos_desc& d) {
  FwdPlan f{};
  const long long S = d.n_segs, Nq = d.n_q_tokens, G = d.n_q_heads / d.n_kv_heads;
  const long long mean_q = (Nq + S - 1) / S, mean_k = (d.n_k_tokens + S - 1) / S;
  long long busy, chunks;  // CTAs with work, about; key chunks of an average segment
  if (mean_q <= 16) {
    const long long gh = G < 16 ? G : 16, t = 16 / gh, hgroups = (G + gh - 1) / gh;
    f.rows = 0;
    f.ctas = (Nq / t + S) * d.n_kv_heads * hgroups;
    busy = ((mean_q + t - 1) / t) * (Nq < S ? Nq : S) * d.n_kv_heads * hgroups;
    chunks = (mean_k + 127) / 128;  // four warps of 32 keys
  } else {
    f.rows = mean_q <= 64 ? 64 : 128;
    f.ctas = (Nq / f.rows + S) * d.n_q_heads;
    busy = ((mean_q + f.rows - 1) / f.rows) * S * d.n_q_heads;
    chunks = (mean_k + 63) / 64;
  }
  const long long want = 3 * kSms, most = chunks / 4;
  long long sp = busy > 0 && busy < want ? want / busy : 1;
  if (sp > most) sp = most;
  if (sp > 64) sp = 64;
  if (sp < 1) sp = 1;
  f.splits = (int)sp;
  f.ctas *= sp;
  return f;
}

inline BwdPlan bwd_plan(const lsrm_relpos_desc& d) {
  BwdPlan b{};
  const long long S = d.n_segs, G = d.n_q_heads / d.n_kv_heads;
  const long long mean_q = (d.n_q_tokens + S - 1) / S, mean_k = (d.n_k_tokens + S - 1) / S;
  b.dq_tiles = d.n_q_tokens / kBwdRows + S;
  b.kv_tiles = d.n_k_tokens / kBwdRows + S;
  const long long busy = ((mean_k + kBwdRows - 1) / kBwdRows) * S * d.n_kv_heads;
  const long long qchunks = (mean_q + 63) / 64, most = G * (qchunks > 0 ? qchunks : 1);
  long long sp = busy > 0 ? (3 * kSms + busy - 1) / busy : 1;
  if (sp < G) {
    while (G % sp) ++sp;  // whole heads, evenly
  } else {
    sp = (sp + G - 1) / G * G;
  }
  if (sp > most) sp = most;
  if (sp > 128) sp = 128;
  b.splits = (int)(sp < 1 ? 1 : sp);
  return b;
}

struct Ws {
  size_t status, o_part, ml_part, delta, corr, tab_part, kv_part, total;
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
  w.tab_part = up256(w.corr + rows * 4);
  w.kv_part = up256(w.tab_part + (size_t)b.dq_tiles * d.n_q_heads * d.n_axes * d.n_buckets * 4);
  const size_t kv = b.splits > 1 ? (size_t)b.splits * 2 * d.n_k_tokens * d.n_kv_heads * D : 0;
  const size_t bwd = up256(w.kv_part + kv * 4);
  w.total = fwd > bwd ? fwd : bwd;
  return w;
}

}  // namespace rp
}  // namespace lsrm
