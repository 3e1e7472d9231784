// Backward of the attention with a learned relative position bias by buckets (relpos.cuh has the
// forward).  With P = exp(t - lse), dP = dO V^T, Delta = sum_j P dP, dS = P (dP - Delta):
//   dq = scale dS K,  dk = scale sum_heads dS^T q,  dv = sum_heads P^T dO,
//   dtable[a][b][h] = sum over the pairs (i, j) of head h with bucket_of[delta_a + D] = b of dS_ij
//
// Two passes over the scores, each with its own tile of rows kept in registers from the scores to
// the products (mma.sync: P and dS go from the accumulator layout to the operand layout in place):
//   * rp_dq_kernel: queries of one head a CTA, keys streaming: dq, and Delta for the other pass;
//   * rp_dkv_kernel: keys of one KV head a CTA, the queries of its heads streaming: dk, dv and the
//     table's gradient.
// Both passes take 64-row tiles and mma.sync: with segments of up to a few hundred tokens, 128-row tiles of
// tcgen05 are half empty (bwd_plan has the measured borders).  Many short segments have a dq pass of their own
// (relpos_short.cu).  What bounds the passes is the per-score work (exponential, look-ups, and in the key pass the
// table's sums: 256 ragged blocks of up to 64 tokens, 32 heads of 32: 134 us at 1.8 warp instructions a clock), not the
// tensor pipe (6%).
//
// Delta.  sum_d dO o with the forward's out is off by that output's bf16 rounding, which a gradient
// that adds up a whole row of dS (the table's) or few keys (short segments) would show.  With D~ that
// value, the row sum of P (dP - D~) is exactly Delta - D~, so the dq pass adds up what it computes
// anyway and hands the exact Delta to the key pass.  Its own dq takes the correction - (Delta - D~) P K, a product
// more: in rows with nearly all weight on one key dS nearly cancels, and without it such a row of dq is off by several
// times its size (512 keys, scores of deviation 8), however many the keys.
//
// The table's gradient: every thread has its own column of NA x buckets sums in shared memory, so
// the sums need no atomics; a tile that lies on one distance adds its sum once (kept in a register
// until the bucket changes), runs of queries on one position add their sums, others score by score.
// CTAs write their sums per (key tile, head) and rp_table_kernel adds them in a fixed order.  dk and dv
// of a key are summed over the heads of its group inside a CTA, or over a fixed number of splits joined
// by rp_dkv_join_kernel in order.  Nothing depends on scheduling: a second run gives the same bits.
//
// Sums are fp32.  P and dS are rounded to bf16 as operands of the products whose other operand is
// bf16; dtable and Delta add the unrounded values.
#include "relpos.cuh"

namespace lsrm {
namespace rp {

constexpr int MT = 1;  // row tiles of 16 a warp: a second one's operands and sums would halve the warps an SM holds
constexpr int kBThreads = 128, kBChunk = 64, kBStages = 3, kKeyStages = 2;

template <int D, int NA>
struct BwdCfg {
  static constexpr int kTile = kBChunk * D / 8;
  static constexpr size_t kRing = (size_t)kBStages * (2 * kTile * 16 + kBChunk * NA * 4);
  static constexpr size_t kKeyRing = (size_t)kKeyStages * (2 * kTile * 16 + kBChunk * (NA * 4 + 8));
  __host__ __device__ static size_t lut(int maxd) { return (((size_t)NA * (2 * maxd + 1) * 4) + 15) & ~(size_t)15; }
  static size_t smem_dq(int maxd) { return kRing + lut(maxd); }
  static size_t smem_dkv(int maxd, int nb) {
    return kKeyRing + lut(maxd) + (size_t)NA * (nb + 1) * kBThreads * 4 +
           ((size_t)2 * maxd + 1) * 4;
  }
};

template <int D, int NA>
__global__ void __launch_bounds__(kBThreads, D == 32 ? 3 : 2) rp_dq_kernel(const Params p) {
  using C = BwdCfg<D, NA>;
  constexpr int kRows = 64 * MT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* ks = reinterpret_cast<uint4*>(smem_raw);
  uint4* vs = ks + kBStages * C::kTile;
  int* ps = reinterpret_cast<int*>(vs + kBStages * C::kTile);
  float* lut = reinterpret_cast<float*>(smem_raw + C::kRing);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  const int h = blockIdx.x % p.Hq, tile = blockIdx.x / p.Hq, hk = h / p.G;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, kRows, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + (tile - first) * kRows;
  if (tile < first || row0 >= qhi) return;
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int nk = khi - klo, chunks = (nk + kBChunk - 1) / kBChunk, top = 2 * p.maxd;

  auto load = [&](int c) {
    if (c < chunks) {
      const int st = c % kBStages, k0 = klo + c * kBChunk, n = min(kBChunk, khi - k0);
      load_tile<D, kBChunk, kBThreads>(ks + st * C::kTile, p.k, k0, n, p.Hkv, hk, tid);
      load_tile<D, kBChunk, kBThreads>(vs + st * C::kTile, p.v, k0, n, p.Hkv, hk, tid);
      for (int i = tid; i < kBChunk * NA; i += kBThreads)
        cp_async4(ps + st * kBChunk * NA + i, p.pos_k + (size_t)(k0 + min(i / NA, n - 1)) * NA + i % NA, true);
    }
    cp_async_commit();
  };
  load(0);
  load(1);
  const bool small = fill_units<NA, kBThreads>(p, lut, h, tid);
  const float mul = small ? p.scale * kLog2e : p.scale;

  uint32_t qa[MT][D / 16][4], da[MT][D / 16][4];
  int qp[MT][2][NA], q_lo[NA], q_hi[NA];
  float delta[MT][2], rest[MT][2], l[MT][2], row[MT][2];
  const int wrow = row0 + warp * 16 * MT;
#pragma unroll
  for (int a = 0; a < NA; ++a) q_lo[a] = INT32_MAX, q_hi[a] = INT32_MIN;
  bool huge = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = wrow + mt * 16 + g;
    const size_t a0 = ((size_t)r * p.Hq + h) * D, a1 = ((size_t)(r + 8) * p.Hq + h) * D;
    const bool l0 = r < qhi, l1 = r + 8 < qhi;
    load_a_rows<D>(qa[mt], l0 ? p.q + a0 : nullptr, l1 ? p.q + a1 : nullptr, lane);
    load_a_rows<D>(da[mt], l0 ? p.dout + a0 : nullptr, l1 ? p.dout + a1 : nullptr, lane);
    uint32_t oa[D / 16][4];
    load_a_rows<D>(oa, l0 ? p.o_in + a0 : nullptr, l1 ? p.o_in + a1 : nullptr, lane);
    delta[mt][0] = delta[mt][1] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = bf16_to_f32((uint16_t)da[mt][d][e]) * bf16_to_f32((uint16_t)oa[d][e]);
        delta[mt][e & 1] +=
            fmaf(__uint_as_float(da[mt][d][e] & 0xffff0000u), __uint_as_float(oa[d][e] & 0xffff0000u), lo);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ri = r + 8 * i;
      delta[mt][i] = quad_sum(delta[mt][i]);
      rest[mt][i] = l[mt][i] = 0.0f;
      const float lse = row_lse(ri < qhi ? p.lse_in[(size_t)ri * p.Hq + h] : INFINITY);
      huge = huge || is_huge(lse);
      row[mt][i] = row_const(lse, small);
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = p.pos_q[(size_t)min(ri, qhi - 1) * NA + a];
        qp[mt][i][a] = p.maxd - x;
        q_lo[a] = min(q_lo[a], x);
        q_hi[a] = max(q_hi[a], x);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    q_lo[a] = __reduce_min_sync(0xffffffffu, q_lo[a]);
    q_hi[a] = __reduce_max_sync(0xffffffffu, q_hi[a]);
    if (q_lo[a] < -kPosLimit || q_hi[a] > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
  }
  const bool exact = !small || __any_sync(0xffffffffu, huge);
  float dq[MT][D / 8][4], pk[MT][D / 8][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dq[mt][n][e] = pk[mt][n][e] = 0.0f;

  for (int c = 0; c < chunks; ++c) {
    cp_async_wait<1>();
    __syncthreads();
    load(c + 2);
    const uint4* kt = ks + (c % kBStages) * C::kTile;
    const uint4* vt = vs + (c % kBStages) * C::kTile;
#pragma unroll 1
    for (int kb = 0; kb < kBChunk; kb += kCols) {
      const int left = nk - c * kBChunk - kb;
      if (left <= 0 || wrow >= qhi) break;
      const int* pt = ps + (c % kBStages) * kBChunk * NA + kb * NA;
      float s[MT][kGroups][4], dp[MT][kGroups][4];
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        uint32_t b[D / 8];
        load_b_rows<D>(b, kt, kb, n, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][n][e] = dp[mt][n][e] = 0.0f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(s[mt][n], qa[mt][d], b + 2 * d);
        }
        load_b_rows<D>(b, vt, kb, n, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(dp[mt][n], da[mt][d], b + 2 * d);
      }
      int mode[NA], one[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a)
        mode[a] = axis_mode<NA>(pt + a, q_lo[a], q_hi[a], false, p.maxd, lane, one[a], p.status);
      float base[MT][2];
      const bool fold = add_bias<NA, MT, 1>(s, base, mode, one, pt, lut, top, qp, mul, exact, tq);
      if (left < kCols) {
        keep_branch();
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (tq * kLaneCols + 2 * n + e >= left)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) s[mt][n][e] = s[mt][n][2 + e] = -INFINITY;
      }
      uint32_t sa[MT][2][4], pa[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float cst = base[mt][i] - row[mt][i];
          float sum0 = 0.0f, sum1 = 0.0f, l0 = 0.0f, l1 = 0.0f;
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            float p0 = s[mt][n][2 * i], p1 = s[mt][n][2 * i + 1];
            if (fold) {
              ffma2(p0, p1, p0, p1, mul, cst);
            } else {  // the subtraction first: exact for scores of any size
              fadd2_acc(p0, p1, -row[mt][i], -row[mt][i]);
              if (!small) fmul2(p0, p1, p0, p1, kLog2e, kLog2e);
            }
            p0 = ex2(p0);
            p1 = ex2(p1);
            fadd2_acc(l0, l1, p0, p1);
            pa[mt][n >> 1][(n & 1) * 2 + i] = pack2(p0, p1);
            float d0 = dp[mt][n][2 * i], d1 = dp[mt][n][2 * i + 1];
            fadd2_acc(d0, d1, -delta[mt][i], -delta[mt][i]);
            fmul2(d0, d1, d0, d1, p0, p1);
            fadd2_acc(sum0, sum1, d0, d1);
            sa[mt][n >> 1][(n & 1) * 2 + i] = pack2(d0, d1);
          }
          rest[mt][i] += sum0 + sum1;
          l[mt][i] += l0 + l1;
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int dc = 0; dc < D / 8; dc += 2) {
          uint32_t b[4];
          load_b_cols<D>(b, kt, kb, j, dc, lane);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(dq[mt][dc], sa[mt][j], b);
            mma16816(dq[mt][dc + 1], sa[mt][j], b + 2);
            mma16816(pk[mt][dc], pa[mt][j], b);
            mma16816(pk[mt][dc + 1], pa[mt][j], b + 2);
          }
        }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sum = quad_sum(l[mt][i]), parts = quad_sum(rest[mt][i]);
      const int r = wrow + mt * 16 + g + 8 * i;
      if (r >= qhi) continue;
      const float inv = row_inverse(sum, row[mt][i], p.status), corr = row_corr(sum);
      const float more = parts * inv, f = inv * p.scale;  // more: Delta - D~
      const size_t at = (size_t)r * p.Hq + h;
      if (tq == 0) {
        p.delta[at] = delta[mt][i] + more;
        p.lse2[at] = row_lse2(row[mt][i], small, corr);
        p.corr[at] = corr;
      }
      uint16_t* to = p.dq + at * D + 2 * tq;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<uint32_t*>(to + n * 8) =
            pack2(fmaf(-more, pk[mt][n][2 * i], dq[mt][n][2 * i]) * f,
                  fmaf(-more, pk[mt][n][2 * i + 1], dq[mt][n][2 * i + 1]) * f);
    }
}

template <int D, int NA>
__global__ void __launch_bounds__(kBThreads, D == 32 ? 4 : 2) rp_dkv_kernel(const Params p) {
  using C = BwdCfg<D, NA>;
  constexpr int kRows = 64 * MT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* qs = reinterpret_cast<uint4*>(smem_raw);
  uint4* ds = qs + kKeyStages * C::kTile;
  int* ps = reinterpret_cast<int*>(ds + kKeyStages * C::kTile);
  float* ls = reinterpret_cast<float*>(ps + kKeyStages * kBChunk * NA);  // [stage][2][chunk]: LSE (log2 units), Delta
  float* lut = ls + kKeyStages * 2 * kBChunk;
  float* hist = lut + C::lut(p.maxd) / 4;  // [NA][NB and one for ids out of range][threads]
  int* boff = reinterpret_cast<int*>(hist + (size_t)NA * (p.NB + 1) * kBThreads);  // a bucket's byte offset

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  const int bins = NA * p.NB;
  let_dependents();
  int unit = blockIdx.x;
  const int split = unit % p.splits;
  unit /= p.splits;
  const int hk = unit % p.Hkv, tile = unit / p.Hkv;
  int first, qlo = 0, qhi = 0, klo, khi;
  const int seg = seg_of_tile(p.off_k, p.S, p.Nk, kRows, tile, first);
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int row0 = klo + (tile - first) * kRows;
  const bool empty = tile < first || row0 >= khi;
  if (!empty) seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int nq = qhi - qlo, chunks = (nq + kBChunk - 1) / kBChunk, top = 2 * p.maxd;
  int h0, h1, c0, c1, part;
  split_range(p, split, chunks, h0, h1, c0, c1, part);
  const int parts = p.splits > p.G ? p.splits / p.G : 1;
  float* tab_part = p.tab_part + (((size_t)tile * parts + part) * p.Hq + hk * p.G) * bins;  // + head * bins
  if (empty) {
    for (int i = h0 * bins + tid; i < h1 * bins; i += kBThreads) tab_part[i] = 0.0f;
    return;
  }
  const int nc = c1 - c0, steps = (h1 - h0) * nc;

  auto load = [&](int it) {
    if (it < steps) {
      const int h = hk * p.G + h0 + it / nc, q0 = qlo + (c0 + it % nc) * kBChunk, n = min(kBChunk, qhi - q0);
      const int st = it % kKeyStages;
      load_tile<D, kBChunk, kBThreads>(qs + st * C::kTile, p.q, q0, n, p.Hq, h, tid);
      load_tile<D, kBChunk, kBThreads>(ds + st * C::kTile, p.dout, q0, n, p.Hq, h, tid);
      for (int i = tid; i < kBChunk * NA; i += kBThreads)
        cp_async4(ps + st * kBChunk * NA + i, p.pos_q + (size_t)(q0 + min(i / NA, n - 1)) * NA + i % NA, true);
      static_assert(kBThreads == 2 * kBChunk, "one row constant a thread");
      cp_async4(ls + st * 2 * kBChunk + tid,
                (tid < kBChunk ? p.lse2 : p.delta) + (size_t)(q0 + min(tid % kBChunk, n - 1)) * p.Hq + h, true);
    }
    cp_async_commit();
  };
  load(0);
  for (int i = tid; i < top + 1; i += kBThreads) {
    const int b = p.bucket_of[i];
    boff[i] = (b < 0 || b >= p.NB ? p.NB : b) * kBThreads * 4;
  }
  for (int b = 0; b < bins + NA; ++b) hist[b * kBThreads + tid] = 0.0f;  // the thread's own column
  char* col = reinterpret_cast<char*>(hist + tid);
  const int axis_bytes = (p.NB + 1) * kBThreads * 4;

  uint32_t ka[MT][D / 16][4], va[MT][D / 16][4];
  int kp[MT][2][NA], k_lo[NA], k_hi[NA];
  const int wrow = row0 + warp * 16 * MT;
#pragma unroll
  for (int a = 0; a < NA; ++a) k_lo[a] = INT32_MAX, k_hi[a] = INT32_MIN;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = wrow + mt * 16 + g;
    const size_t a0 = ((size_t)r * p.Hkv + hk) * D, a1 = ((size_t)(r + 8) * p.Hkv + hk) * D;
    load_a_rows<D>(ka[mt], r < khi ? p.k + a0 : nullptr, r + 8 < khi ? p.k + a1 : nullptr, lane);
    load_a_rows<D>(va[mt], r < khi ? p.v + a0 : nullptr, r + 8 < khi ? p.v + a1 : nullptr, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = p.pos_k[(size_t)min(r + 8 * i, khi - 1) * NA + a];
        kp[mt][i][a] = p.maxd + x;
        k_lo[a] = min(k_lo[a], x);
        k_hi[a] = max(k_hi[a], x);
      }
  }
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    k_lo[a] = __reduce_min_sync(0xffffffffu, k_lo[a]);
    k_hi[a] = __reduce_max_sync(0xffffffffu, k_hi[a]);
  }
  float dk[MT][D / 8][4], dv[MT][D / 8][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dk[mt][n][e] = dv[mt][n][e] = 0.0f;
  // the running sum of tiles on one distance, and its bucket
  float run[NA];
  int run_b[NA];
#pragma unroll
  for (int a = 0; a < NA; ++a) run[a] = 0.0f, run_b[a] = p.NB * kBThreads * 4;
  // the head's sums of the CTA's threads to global memory, and the columns back to 0
  auto flush = [&](int head) {
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      *reinterpret_cast<float*>(col + a * axis_bytes + run_b[a]) += run[a];
      run[a] = 0.0f;
    }
    __syncthreads();
    flush_sums<kBThreads, kBThreads>(hist, bins, p.NB, tid, tab_part + head * bins);
    __syncthreads();
  };

  bool small = false;
  float mul = 0.0f;
  for (int it = 0; it < steps; ++it) {
    const int head = h0 + it / nc, cc = it % nc;
    cp_async_wait<0>();
    __syncthreads();
    load(it + 1);
    if (cc == 0) {  // the barriers since the last head's tiles ended the old table's use
      small = fill_units<NA, kBThreads>(p, lut, hk * p.G + head, tid);
      mul = small ? p.scale * kLog2e : p.scale;
    }
    const int st = it % kKeyStages;
    const uint4* qt = qs + st * C::kTile;
    const uint4* dt = ds + st * C::kTile;
    const float* lc = ls + st * 2 * kBChunk;
    const bool exact = !small || __any_sync(0xffffffffu, is_huge(lc[lane]) || is_huge(lc[lane + 32]));
#pragma unroll 1
    for (int qb = 0; qb < kBChunk; qb += kCols) {
      const int left = nq - (c0 + cc) * kBChunk - qb;
      if (left <= 0 || wrow >= khi) break;
      const int* pt = ps + st * kBChunk * NA + qb * NA;
      const float* lt = ls + st * 2 * kBChunk + qb + tq * kLaneCols;
      float s[MT][kGroups][4], dp[MT][kGroups][4];
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        uint32_t b[D / 8];
        load_b_rows<D>(b, qt, qb, n, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][n][e] = dp[mt][n][e] = 0.0f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(s[mt][n], ka[mt][d], b + 2 * d);
        }
        load_b_rows<D>(b, dt, qb, n, lane);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(dp[mt][n], va[mt][d], b + 2 * d);
      }
      int mode[NA], one[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a)
        mode[a] = axis_mode<NA>(pt + a, k_lo[a], k_hi[a], true, p.maxd, lane, one[a], p.status);
      float base[MT][2];
      const bool fold = add_bias<NA, MT, -1>(s, base, mode, one, pt, lut, top, kp, mul, exact, tq);
      bool flat = true;  // one bias for the tile
#pragma unroll
      for (int a = 0; a < NA; ++a) flat = flat && mode[a] == kOne;
      // s becomes dS^T, dp becomes P^T
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        float2 l = *reinterpret_cast<const float2*>(lt + 2 * n);
        const float2 dl = *reinterpret_cast<const float2*>(lt + kBChunk + 2 * n);
        if (left < kCols) {  // no query: P = 0
          keep_branch();
          if (tq * kLaneCols + 2 * n >= left) l.x = INFINITY;
          if (tq * kLaneCols + 2 * n + 1 >= left) l.y = INFINITY;
        }
        if (!exact) {
          if (fold) {
            const float c0 = flat ? base[0][0] - l.x : -l.x, c1 = flat ? base[0][0] - l.y : -l.y;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float d0 = c0, d1 = c1;
                if (!flat) fadd2_acc(d0, d1, base[mt][i], base[mt][i]);
                ffma2v(s[mt][n][2 * i], s[mt][n][2 * i + 1], s[mt][n][2 * i], s[mt][n][2 * i + 1], mul, d0, d1);
              }
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i) fadd2_acc(s[mt][n][2 * i], s[mt][n][2 * i + 1], -l.x, -l.y);
          }
        } else {
          // the row's constant and the correction one after the other: together they would be rounded to the former's
          // spacing
          keep_branch();
          float ln[2], cr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool there = tq * kLaneCols + 2 * n + e < left;
            const int col = there ? tq * kLaneCols + 2 * n + e : 0;
            const size_t at = (size_t)(qlo + (c0 + cc) * kBChunk + qb + col) * p.Hq + hk * p.G + head;
            ln[e] = row_const(there ? row_lse(p.lse_in[at]) : INFINITY, small);
            cr[e] = there ? p.corr[at] : 0.0f;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = s[mt][n][2 * i + e] - ln[e];
                s[mt][n][2 * i + e] = small ? x - cr[e] : fmaf(x, kLog2e, -cr[e]);
              }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p0 = ex2(s[mt][n][2 * i]), p1 = ex2(s[mt][n][2 * i + 1]);
            float d0 = dp[mt][n][2 * i], d1 = dp[mt][n][2 * i + 1];
            fadd2_acc(d0, d1, -dl.x, -dl.y);
            fmul2(s[mt][n][2 * i], s[mt][n][2 * i + 1], d0, d1, p0, p1);
            dp[mt][n][2 * i] = p0;
            dp[mt][n][2 * i + 1] = p1;
          }
      }
      if (wrow + 16 * MT > khi) {  // rows past the segment's last key have no pairs
        keep_branch();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (wrow + mt * 16 + g + 8 * i >= khi)
#pragma unroll
              for (int n = 0; n < kGroups; ++n) s[mt][n][2 * i] = s[mt][n][2 * i + 1] = 0.0f;
      }
      // the table's gradient
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        char* ca = col + a * axis_bytes;
        if (mode[a] == kOne) {
          const int b = boff[one[a]];
          if (b != run_b[a]) {
            *reinterpret_cast<float*>(ca + run_b[a]) += run[a];
            run[a] = 0.0f;
            run_b[a] = b;
          }
          float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < kGroups; ++n) {
              fadd2_acc(sum0, sum1, s[mt][n][0], s[mt][n][1]);
              fadd2_acc(sum0, sum1, s[mt][n][2], s[mt][n][3]);
            }
          run[a] += sum0 + sum1;
        } else if (mode[a] <= kFour) {
          // runs of eight or four queries on one position
          const int x0 = -pt[tq * kLaneCols * NA + a], x1 = -pt[(tq * kLaneCols + 4) * NA + a];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              add_two(ca, boff[clamp_index(x0, kp[mt][i][a], top)],
                      (s[mt][0][2 * i] + s[mt][0][2 * i + 1]) + (s[mt][1][2 * i] + s[mt][1][2 * i + 1]),
                      boff[clamp_index(x1, kp[mt][i][a], top)],
                      (s[mt][2][2 * i] + s[mt][2][2 * i + 1]) + (s[mt][3][2 * i] + s[mt][3][2 * i + 1]));
        } else if (mode[a] == kTurn) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int x0 = -pt[(tq * kLaneCols + 2 * n) * NA + a], x1 = -pt[(tq * kLaneCols + 2 * n + 1) * NA + a];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                add_two(ca, boff[clamp_index(x0, kp[mt][i][a], top)], s[mt][n][2 * i] + s[mt][n + 2][2 * i],
                        boff[clamp_index(x1, kp[mt][i][a], top)], s[mt][n][2 * i + 1] + s[mt][n + 2][2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            const int x0 = -pt[(tq * kLaneCols + 2 * n) * NA + a], x1 = -pt[(tq * kLaneCols + 2 * n + 1) * NA + a];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                add_two(ca, boff[clamp_index(x0, kp[mt][i][a], top)], s[mt][n][2 * i],
                        boff[clamp_index(x1, kp[mt][i][a], top)], s[mt][n][2 * i + 1]);
          }
        }
      }
      uint32_t sa[MT][2][4], pa[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sa[mt][n >> 1][(n & 1) * 2 + i] = pack2(s[mt][n][2 * i], s[mt][n][2 * i + 1]);
            pa[mt][n >> 1][(n & 1) * 2 + i] = pack2(dp[mt][n][2 * i], dp[mt][n][2 * i + 1]);
          }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int dc = 0; dc < D / 8; dc += 2) {
          uint32_t b[4];
          load_b_cols<D>(b, qt, qb, j, dc, lane);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(dk[mt][dc], sa[mt][j], b);
            mma16816(dk[mt][dc + 1], sa[mt][j], b + 2);
          }
          load_b_cols<D>(b, dt, qb, j, dc, lane);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(dv[mt][dc], pa[mt][j], b);
            mma16816(dv[mt][dc + 1], pa[mt][j], b + 2);
          }
        }
    }
    if (cc == nc - 1) flush(head);
  }
  if (steps == 0)  // no query: the table's sums are 0
    for (int i = h0 * bins + tid; i < h1 * bins; i += kBThreads) tab_part[i] = 0.0f;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = wrow + mt * 16 + g + 8 * i;
      if (r >= khi) continue;
      const size_t at = ((size_t)r * p.Hkv + hk) * D + 2 * tq;
      if (p.splits == 1) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          *reinterpret_cast<uint32_t*>(p.dk + at + n * 8) =
              pack2(dk[mt][n][2 * i] * p.scale, dk[mt][n][2 * i + 1] * p.scale);
          *reinterpret_cast<uint32_t*>(p.dv + at + n * 8) = pack2(dv[mt][n][2 * i], dv[mt][n][2 * i + 1]);
        }
      } else {
        const size_t stride = (size_t)p.Nk * p.Hkv * D;
        float* to = p.kv_part + (size_t)split * 2 * stride + at;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          *reinterpret_cast<float2*>(to + n * 8) = make_float2(dk[mt][n][2 * i], dk[mt][n][2 * i + 1]);
          *reinterpret_cast<float2*>(to + stride + n * 8) = make_float2(dv[mt][n][2 * i], dv[mt][n][2 * i + 1]);
        }
      }
    }
}

// dtable = the tiles' sums in order: 32 bins a CTA, 32 runs of tiles, joined in shared memory
__global__ void __launch_bounds__(1024) rp_table_kernel(const Params p, int tiles, int bins) {
  __shared__ float part[32][33];
  wait_for_previous();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, h = blockIdx.y, b = blockIdx.x * 32 + lane;
  float x = 0.0f;
  if (b < bins) {
#pragma unroll 4
    for (int t = run; t < tiles; t += 32) x += p.tab_part[((size_t)t * p.Hq + h) * bins + b];
  }
  part[run][lane] = x;
  __syncthreads();
  if (run != 0 || b >= bins) return;
  x = 0.0f;
#pragma unroll
  for (int r = 0; r < 32; ++r) x += part[r][lane];
  p.dtable[(size_t)b * p.Hq + h] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

constexpr int kSumRows = 8, kSumThreads = 256;

// dk = scale x the splits' sums in order, dv likewise without the scale; only rows of segments
template <int D>
__global__ void __launch_bounds__(kSumThreads) rp_dkv_join_kernel(const Params p) {
  int first, klo, khi;
  const int seg = seg_of_tile(p.off_k, p.S, p.Nk, kSumRows, blockIdx.x, first);
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int row0 = klo + ((int)blockIdx.x - first) * kSumRows;
  wait_for_previous();
  let_dependents();
  if ((int)blockIdx.x < first || row0 >= khi) return;
  const int n = min(kSumRows, khi - row0) * p.Hkv * D / 4;
  const size_t stride = (size_t)p.Nk * p.Hkv * D;
  for (int i = threadIdx.x; i < 2 * n; i += kSumThreads) {
    const bool is_v = i >= n;
    const size_t at = (size_t)row0 * p.Hkv * D + (size_t)(is_v ? i - n : i) * 4;
    const float* src = p.kv_part + (is_v ? stride : 0) + at;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      const float4 y = *reinterpret_cast<const float4*>(src + (size_t)s * 2 * stride);
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    const float f = is_v ? 1.0f : p.scale;
    *reinterpret_cast<uint2*>((is_v ? p.dv : p.dk) + at) =
        make_uint2(pack2(x.x * f, x.y * f), pack2(x.z * f, x.w * f));
  }
}

static lsrm_status launched() { return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA; }

template <int D, int NA>
static lsrm_status run_dq(const Params& p, const BwdPlan& b, cudaStream_t s) {
  const size_t bytes = BwdCfg<D, NA>::smem_dq(p.maxd);
  if (!allow_smem(rp_dq_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
  rp_dq_kernel<D, NA><<<(unsigned)(b.dq_tiles * p.Hq), kBThreads, bytes, s>>>(p);
  return launched();
}
template <int D, int NA>
static lsrm_status run_dkv(const Params& p, const BwdPlan& b, cudaStream_t s) {
  const size_t bytes = BwdCfg<D, NA>::smem_dkv(p.maxd, p.NB);
  if (!allow_smem(rp_dkv_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
  rp_dkv_kernel<D, NA><<<(unsigned)(b.kv_tiles * p.Hkv * p.splits), kBThreads, bytes, s>>>(p);
  return launched();
}

lsrm_status launch_bwd_tc(const Params& p, int D, int NA, const BwdPlan& b, cudaStream_t s);
lsrm_status launch_short(const Params& p, int D, int NA, long long ctas, bool dq, cudaStream_t s);

template <int D, int NA>
static lsrm_status run_bwd(const Params& p, const BwdPlan& b, cudaStream_t s) {
  lsrm_status st = LSRM_OK;
  if (b.tc) {
    if ((st = launch_bwd_tc(p, D, NA, b, s)) != LSRM_OK) return st;
  }
  if (!b.tc && p.Nq > 0) {
    st = b.shrt ? launch_short(p, D, NA, b.short_ctas, true, s) : run_dq<D, NA>(p, b, s);
    if (st != LSRM_OK) return st;
  }
  if (p.Nk > 0) {
    if (!b.tc && (st = run_dkv<D, NA>(p, b, s)) != LSRM_OK) return st;
    if (p.splits > 1) {
      if (!launch_dependent(rp_dkv_join_kernel<D>, dim3((unsigned)(p.Nk / kSumRows + p.S)), kSumThreads, s, p))
        return LSRM_ERR_CUDA;
    }
  }
  const int bins = NA * p.NB;
  const int tiles = p.Nk > 0 ? (int)(b.kv_tiles * b.parts()) : 0;
  return launch_dependent(rp_table_kernel, dim3((unsigned)((bins + 31) / 32), (unsigned)p.Hq), 1024, s, p, tiles, bins)
             ? LSRM_OK
             : LSRM_ERR_CUDA;
}

}  // namespace rp

lsrm_status launch_relpos_backward(const rp::Params& p, int D, int NA, const rp::BwdPlan& b, cudaStream_t s) {
  using namespace rp;
  if (D == 32) {
    if (NA == 1) return run_bwd<32, 1>(p, b, s);
    if (NA == 2) return run_bwd<32, 2>(p, b, s);
    return run_bwd<32, 3>(p, b, s);
  }
  if (NA == 1) return run_bwd<64, 1>(p, b, s);
  if (NA == 2) return run_bwd<64, 2>(p, b, s);
  return run_bwd<64, 3>(p, b, s);
}

}  // namespace lsrm
