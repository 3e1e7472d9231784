// Backward of the attention with a learned relative position bias by buckets (relpos.cuh has the
// forward).  With P = exp(t - lse), dP = dO V^T, Delta = sum_d dO o, dS = P (dP - Delta):
//   dq = scale dS K,  dk = scale sum_heads dS^T q,  dv = sum_heads P^T dO,
//   dtable[a][b][h] = sum over the pairs (i, j) of head h with bucket_of[delta_a + D] = b of dS_ij
//
// Two passes over the scores, each with its own tile of rows kept in registers from the scores to
// the products (mma.sync: P and dS go from the accumulator layout to the operand layout in place):
//   * rp_dq_kernel: 64 queries of one head a CTA, keys streaming: dq and the table's gradient.
//   * rp_dkv_kernel: 64 keys of one KV head a CTA, the queries of its heads streaming: dk, dv.
//
// The table's gradient: every thread has its own column of NA x buckets sums in shared memory, so
// the sums need no atomics; a tile that lies on one distance adds its sum once (kept in a register
// until the bucket changes), other tiles add score by score.  CTAs write their sums per (query tile,
// head) and rp_table_kernel adds them in a fixed order.  dk and dv of a key are summed over the heads
// of its group inside a CTA, or over a fixed number of splits joined by rp_dkv_join_kernel in order.
// Nothing depends on scheduling: a second run gives the same bits.
//
// Sums are fp32.  P and dS are rounded to bf16 as operands of the products whose other operand is
// bf16; dtable adds the unrounded dS.
#include "relpos.cuh"

namespace lsrm {
namespace rp {

constexpr int kBThreads = 128, kBChunk = 64, kBStages = 3;

template <int D, int NA>
struct BwdCfg {
  static constexpr int kTile = kBChunk * D / 8;
  static constexpr size_t kRing = (size_t)kBStages * (2 * kTile * 16 + kBChunk * NA * 4);
  __host__ __device__ static size_t lut(int maxd) { return (((size_t)NA * (2 * maxd + 1) * 4) + 15) & ~(size_t)15; }
  static size_t smem_dq(int maxd, int nb) {
    return kRing + lut(maxd) + (size_t)NA * nb * kBThreads * 4 + (((size_t)2 * maxd + 1 + 15) & ~(size_t)15);
  }
  static size_t smem_dkv(int maxd) { return kRing + (size_t)kBStages * kBChunk * 12 + lut(maxd); }
};

// Rows whose |LSE| is so large that fp32 lost the logarithm of their sum beside the largest score
// (every key masked by a huge finite bias): corr = log2 sum_j exp(t - lse), a row at a time, lanes over
// keys.  The warp's rows are wrow .. wrow + 15; lane (g, .) holds the LSE of rows g and g + 8.
template <int D, int NA>
__device__ __noinline__ void huge_rows(const Params& p, const float* lut, const float* lse, float* corr, int wrow,
                                       int h, int hk, int klo, int khi, int lane) {
  for (int r = 0; r < 16; ++r) {
    const float l = __shfl_sync(0xffffffffu, lse[r >> 3], (r & 7) * 4);
    if (!(fabsf(l) >= kFoldLimit) || l == INFINITY) continue;
    const size_t row = wrow + r;
    const uint16_t* q = p.q + (row * p.Hq + h) * D;
    float sum = 0.0f;
    for (int j = klo + lane; j < khi; j += 32) {
      const uint16_t* k = p.k + ((size_t)j * p.Hkv + hk) * D;
      float t = 0.0f;
      for (int d = 0; d < D; ++d) t = fmaf(bf16_to_f32(q[d]), bf16_to_f32(k[d]), t);
      t *= p.scale;
      for (int a = 0; a < NA; ++a)
        t += lut[a * (2 * p.maxd + 1) + clamp_index(p.pos_k[(size_t)j * NA + a], p.maxd - p.pos_q[row * NA + a],
                                                    2 * p.maxd)];
      sum += fast_exp2((t - l) * kLog2e);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((lane >> 2) == (r & 7)) corr[r >> 3] = log2f(sum);
  }
}

template <int D, int NA>
__global__ void __launch_bounds__(kBThreads) rp_dq_kernel(const Params p) {
  using C = BwdCfg<D, NA>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* ks = reinterpret_cast<uint4*>(smem_raw);
  uint4* vs = ks + kBStages * C::kTile;
  int* ps = reinterpret_cast<int*>(vs + kBStages * C::kTile);
  float* lut = reinterpret_cast<float*>(smem_raw + C::kRing);
  float* hist = reinterpret_cast<float*>(smem_raw + C::kRing + C::lut(p.maxd));  // [NA * NB][threads]
  uint8_t* bk = reinterpret_cast<uint8_t*>(hist + (size_t)NA * p.NB * kBThreads);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  const int h = blockIdx.x % p.Hq, tile = blockIdx.x / p.Hq, hk = h / p.G, bins = NA * p.NB;
  float* tab_part = p.tab_part + (size_t)blockIdx.x * bins;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, kBwdRows, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + (tile - first) * kBwdRows;
  if (tile < first || row0 >= qhi) {
    for (int i = tid; i < bins; i += kBThreads) tab_part[i] = 0.0f;
    return;
  }
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
  fill_lut<NA>(p, lut, h, tid, kBThreads);
  for (int i = tid; i < top + 1; i += kBThreads) {
    const int b = p.bucket_of[i];
    bk[i] = (uint8_t)(b < 0 || b >= p.NB ? 255 : b);
  }
  for (int b = 0; b < bins; ++b) hist[b * kBThreads + tid] = 0.0f;  // the thread's own column

  uint32_t qa[D / 16][4], da[D / 16][4];
  int qp[2][NA], q_lo[NA], q_hi[NA];
  float lse[2], delta[2], corr[2];
  const int wrow = row0 + warp * 16;
  {
    const uint16_t *q0 = nullptr, *q1 = nullptr, *d0 = nullptr, *d1 = nullptr, *o0 = nullptr, *o1 = nullptr;
    const int r = wrow + g;
    const size_t a0 = ((size_t)r * p.Hq + h), a1 = ((size_t)(r + 8) * p.Hq + h);
    if (r < qhi) q0 = p.q + a0 * D, d0 = p.dout + a0 * D, o0 = p.o_in + a0 * D;
    if (r + 8 < qhi) q1 = p.q + a1 * D, d1 = p.dout + a1 * D, o1 = p.o_in + a1 * D;
    load_a_rows<D>(qa, q0, q1, lane);
    load_a_rows<D>(da, d0, d1, lane);
    uint32_t oa[D / 16][4];
    load_a_rows<D>(oa, o0, o1, lane);
    delta[0] = delta[1] = 0.0f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = bf16_to_f32((uint16_t)da[d][e]) * bf16_to_f32((uint16_t)oa[d][e]);
        delta[e & 1] += fmaf(__uint_as_float(da[d][e] & 0xffff0000u), __uint_as_float(oa[d][e] & 0xffff0000u), lo);
      }
#pragma unroll
    for (int a = 0; a < NA; ++a) q_lo[a] = INT32_MAX, q_hi[a] = INT32_MIN;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ri = r + 8 * i;
      const size_t at = (size_t)ri * p.Hq + h;
      delta[i] = quad_sum(delta[i]);
      lse[i] = ri < qhi ? p.lse_in[at] : INFINITY;
      if (lse[i] == -INFINITY) lse[i] = INFINITY;  // a row without keys: P = 0
      if (ri < qhi && tq == 0) p.delta[at] = delta[i];
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = p.pos_q[(size_t)min(ri, qhi - 1) * NA + a];
        qp[i][a] = p.maxd - x;
        q_lo[a] = min(q_lo[a], x);
        q_hi[a] = max(q_hi[a], x);
      }
    }
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      q_lo[a] = __reduce_min_sync(0xffffffffu, q_lo[a]);
      q_hi[a] = __reduce_max_sync(0xffffffffu, q_hi[a]);
      if (q_lo[a] < -kPosLimit || q_hi[a] > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
    }
  }
  __syncthreads();  // the bias table
  corr[0] = corr[1] = 0.0f;
  if (__any_sync(0xffffffffu, (fabsf(lse[0]) >= kFoldLimit && lse[0] != INFINITY) ||
                                  (fabsf(lse[1]) >= kFoldLimit && lse[1] != INFINITY)))
    huge_rows<D, NA>(p, lut, lse, corr, wrow, h, hk, klo, khi, lane);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ri = wrow + g + 8 * i;
    if (ri < qhi && tq == 0) p.corr[(size_t)ri * p.Hq + h] = corr[i];
  }
  float dq[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dq[n][e] = 0.0f;
  // the running sum of tiles on one distance, and its bucket
  float run[NA];
  int run_b[NA];
#pragma unroll
  for (int a = 0; a < NA; ++a) run[a] = 0.0f, run_b[a] = 255;

  for (int c = 0; c < chunks; ++c) {
    cp_async_wait<1>();
    __syncthreads();
    load(c + 2);
    const uint4* kt = ks + (c % kBStages) * C::kTile;
    const uint4* vt = vs + (c % kBStages) * C::kTile;
    const int* pt = ps + (c % kBStages) * kBChunk * NA;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const int kb = half * 32, left = nk - c * kBChunk - kb;
      if (left <= 0 || wrow >= qhi) break;
      float s[4][4], dp[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t b[D / 8];
        load_b_rows<D>(b, kt, kb + n * 8, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = dp[n][e] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) mma_bf16_16816(s[n], qa[d], b + 2 * d);
        load_b_rows<D>(b, vt, kb + n * 8, lane);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) mma_bf16_16816(dp[n], da[d], b + 2 * d);
      }
      int uni[NA];
      bool all_uni = true;
      float ub = 0.0f;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = pt[(kb + lane) * NA + a];
        const int lo = __reduce_min_sync(0xffffffffu, x), hi = __reduce_max_sync(0xffffffffu, x);
        if (lo < -kPosLimit || hi > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
        uni[a] = uniform_index(lo, hi, q_lo[a], q_hi[a], p.maxd);
        all_uni = all_uni && uni[a] >= 0;
        if (uni[a] >= 0) ub += lut[a * (top + 1) + uni[a]];
      }
      all_uni = all_uni && fabsf(ub) < kFoldLimit;
      if (!all_uni) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = fmaf(s[n][e], p.scale, ub);
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          if (uni[a] >= 0) continue;
          const float* la = lut + a * (top + 1);
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int x = pt[(kb + n * 8 + 2 * tq + e) * NA + a];
#pragma unroll
              for (int i = 0; i < 2; ++i) s[n][2 * i + e] += la[clamp_index(x, qp[i][a], top)];
            }
        }
      }
      // s becomes dS
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = p.scale * kLog2e, cst = fmaf(ub - lse[i], kLog2e, -corr[i]);
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float t = s[n][2 * i + e];
            const float pr = fast_exp2(all_uni ? fmaf(t, x, cst) : fmaf(t - lse[i], kLog2e, -corr[i]));
            s[n][2 * i + e] = pr * (dp[n][2 * i + e] - delta[i]);
          }
      }
      if (left < 32) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (n * 8 + 2 * tq + e >= left) s[n][e] = s[n][2 + e] = 0.0f;
      }
      // the table's gradient
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        if (uni[a] >= 0) {
          const int b = bk[uni[a]];
          if (b != run_b[a]) {
            if (run_b[a] != 255) hist[(a * p.NB + run_b[a]) * kBThreads + tid] += run[a];
            run[a] = 0.0f;
            run_b[a] = b;
          }
          float sum = 0.0f;
#pragma unroll
          for (int n = 0; n < 4; ++n) sum += (s[n][0] + s[n][1]) + (s[n][2] + s[n][3]);
          run[a] += sum;
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int x = pt[(kb + n * 8 + 2 * tq + e) * NA + a];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int b = bk[clamp_index(x, qp[i][a], top)];
                if (b != 255) hist[(a * p.NB + b) * kBThreads + tid] += s[n][2 * i + e];
              }
            }
        }
      }
      uint32_t sa[2][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) sa[n >> 1][(n & 1) * 2 + i] = pack_bf16x2(s[n][2 * i], s[n][2 * i + 1]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int dc = 0; dc < D / 8; dc += 2) {
          uint32_t b[4];
          load_b_cols<D>(b, kt, kb + j * 16, dc, lane);
          mma_bf16_16816(dq[dc], sa[j], b);
          mma_bf16_16816(dq[dc + 1], sa[j], b + 2);
        }
    }
  }
#pragma unroll
  for (int a = 0; a < NA; ++a)
    if (run_b[a] != 255) hist[(a * p.NB + run_b[a]) * kBThreads + tid] += run[a];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = wrow + g + 8 * i;
    if (r >= qhi) continue;
    uint16_t* to = p.dq + ((size_t)r * p.Hq + h) * D + 2 * tq;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<uint32_t*>(to + n * 8) = pack_bf16x2(dq[n][2 * i] * p.scale, dq[n][2 * i + 1] * p.scale);
  }
  __syncthreads();
  for (int b = warp; b < bins; b += kBThreads / 32) {
    float x = 0.0f;
#pragma unroll
    for (int t = 0; t < kBThreads; t += 32) x += hist[b * kBThreads + t + lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == 0) tab_part[b] = x;
  }
}

// dtable = the tiles' sums in order: 32 bins a CTA, 32 runs of tiles, joined in shared memory
__global__ void __launch_bounds__(1024) rp_table_kernel(const Params p, int tiles, int bins) {
  __shared__ float part[32][33];
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

template <int D, int NA>
__global__ void __launch_bounds__(kBThreads) rp_dkv_kernel(const Params p) {
  using C = BwdCfg<D, NA>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* qs = reinterpret_cast<uint4*>(smem_raw);
  uint4* ds = qs + kBStages * C::kTile;
  int* ps = reinterpret_cast<int*>(ds + kBStages * C::kTile);
  float* ls = reinterpret_cast<float*>(smem_raw + C::kRing);  // [stage][3][chunk]: LSE, Delta, corr
  float* lut = ls + kBStages * 3 * kBChunk;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  int unit = blockIdx.x;
  const int split = unit % p.splits;
  unit /= p.splits;
  const int hk = unit % p.Hkv, tile = unit / p.Hkv;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_k, p.S, p.Nk, kBwdRows, tile, first);
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int row0 = klo + (tile - first) * kBwdRows;
  if (tile < first || row0 >= khi) return;
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int nq = qhi - qlo, chunks = (nq + kBChunk - 1) / kBChunk, top = 2 * p.maxd;
  // the (head, query chunk) steps of this split, head by head
  const long long total = (long long)p.G * chunks, per = (total + p.splits - 1) / p.splits;
  const int i0 = (int)min(split * per, total), i1 = (int)min(i0 + per, total);

  auto load = [&](int it) {
    if (it < i1) {
      const int h = hk * p.G + it / chunks, q0 = qlo + it % chunks * kBChunk, n = min(kBChunk, qhi - q0);
      const int st = it % kBStages;
      load_tile<D, kBChunk, kBThreads>(qs + st * C::kTile, p.q, q0, n, p.Hq, h, tid);
      load_tile<D, kBChunk, kBThreads>(ds + st * C::kTile, p.dout, q0, n, p.Hq, h, tid);
      for (int i = tid; i < kBChunk * NA; i += kBThreads)
        cp_async4(ps + st * kBChunk * NA + i, p.pos_q + (size_t)(q0 + min(i / NA, n - 1)) * NA + i % NA, true);
      for (int i = tid; i < 3 * kBChunk; i += kBThreads) {
        const float* src = i < kBChunk ? p.lse_in : i < 2 * kBChunk ? p.delta : p.corr;
        cp_async4(ls + st * 3 * kBChunk + i, src + (size_t)(q0 + min(i % kBChunk, n - 1)) * p.Hq + h, true);
      }
    }
    cp_async_commit();
  };
  load(i0);
  load(i0 + 1);

  uint32_t ka[D / 16][4], va[D / 16][4];
  int kp[2][NA], k_lo[NA], k_hi[NA];
  const int wrow = row0 + warp * 16;
  {
    const int r = wrow + g;
    const size_t a0 = ((size_t)r * p.Hkv + hk) * D, a1 = ((size_t)(r + 8) * p.Hkv + hk) * D;
    load_a_rows<D>(ka, r < khi ? p.k + a0 : nullptr, r + 8 < khi ? p.k + a1 : nullptr, lane);
    load_a_rows<D>(va, r < khi ? p.v + a0 : nullptr, r + 8 < khi ? p.v + a1 : nullptr, lane);
#pragma unroll
    for (int a = 0; a < NA; ++a) k_lo[a] = INT32_MAX, k_hi[a] = INT32_MIN;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = p.pos_k[(size_t)min(r + 8 * i, khi - 1) * NA + a];
        kp[i][a] = p.maxd + x;
        k_lo[a] = min(k_lo[a], x);
        k_hi[a] = max(k_hi[a], x);
      }
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      k_lo[a] = __reduce_min_sync(0xffffffffu, k_lo[a]);
      k_hi[a] = __reduce_max_sync(0xffffffffu, k_hi[a]);
    }
  }
  float dk[D / 8][4], dv[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[n][e] = dv[n][e] = 0.0f;

  int head = -1;
  for (int it = i0; it < i1; ++it) {
    cp_async_wait<1>();
    __syncthreads();
    load(it + 2);
    if (it / chunks != head) {  // the same for the whole CTA; the barrier above ended the old table's use
      head = it / chunks;
      fill_lut<NA>(p, lut, hk * p.G + head, tid, kBThreads);
      __syncthreads();
    }
    const int st = it % kBStages;
    const uint4* qt = qs + st * C::kTile;
    const uint4* dt = ds + st * C::kTile;
    const int* pt = ps + st * kBChunk * NA;
    const float* lt = ls + st * 3 * kBChunk;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const int qb = half * 32, left = nq - it % chunks * kBChunk - qb;
      if (left <= 0 || wrow >= khi) break;
      float s[4][4], dp[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t b[D / 8];
        load_b_rows<D>(b, qt, qb + n * 8, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = dp[n][e] = 0.0f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) mma_bf16_16816(s[n], ka[d], b + 2 * d);
        load_b_rows<D>(b, dt, qb + n * 8, lane);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) mma_bf16_16816(dp[n], va[d], b + 2 * d);
      }
      int uni[NA];
      bool all_uni = true;
      float ub = 0.0f;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = pt[(qb + lane) * NA + a];
        uni[a] = uniform_index(k_lo[a], k_hi[a], __reduce_min_sync(0xffffffffu, x),
                               __reduce_max_sync(0xffffffffu, x), p.maxd);
        all_uni = all_uni && uni[a] >= 0;
        if (uni[a] >= 0) ub += lut[a * (top + 1) + uni[a]];
      }
      all_uni = all_uni && fabsf(ub) < kFoldLimit;
      if (!all_uni) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = fmaf(s[n][e], p.scale, ub);
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          if (uni[a] >= 0) continue;
          const float* la = lut + a * (top + 1);
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int x = -pt[(qb + n * 8 + 2 * tq + e) * NA + a];
#pragma unroll
              for (int i = 0; i < 2; ++i) s[n][2 * i + e] += la[clamp_index(x, kp[i][a], top)];
            }
        }
      }
      // s becomes dS^T, dp becomes P^T
      const float x = p.scale * kLog2e;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = n * 8 + 2 * tq + e;
          float lse = lt[qb + col];
          const float delta = lt[kBChunk + qb + col], corr = lt[2 * kBChunk + qb + col];
          if (lse == -INFINITY || col >= left) lse = INFINITY;  // no key, or no query: P = 0
          const float cst = fmaf(ub - lse, kLog2e, -corr);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = s[n][2 * i + e];
            const float pr = fast_exp2(all_uni ? fmaf(t, x, cst) : fmaf(t - lse, kLog2e, -corr));
            s[n][2 * i + e] = pr * (dp[n][2 * i + e] - delta);
            dp[n][2 * i + e] = pr;
          }
        }
      uint32_t sa[2][4], pa[2][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sa[n >> 1][(n & 1) * 2 + i] = pack_bf16x2(s[n][2 * i], s[n][2 * i + 1]);
          pa[n >> 1][(n & 1) * 2 + i] = pack_bf16x2(dp[n][2 * i], dp[n][2 * i + 1]);
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int dc = 0; dc < D / 8; dc += 2) {
          uint32_t b[4];
          load_b_cols<D>(b, qt, qb + j * 16, dc, lane);
          mma_bf16_16816(dk[dc], sa[j], b);
          mma_bf16_16816(dk[dc + 1], sa[j], b + 2);
          load_b_cols<D>(b, dt, qb + j * 16, dc, lane);
          mma_bf16_16816(dv[dc], pa[j], b);
          mma_bf16_16816(dv[dc + 1], pa[j], b + 2);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = wrow + g + 8 * i;
    if (r >= khi) continue;
    const size_t at = ((size_t)r * p.Hkv + hk) * D + 2 * tq;
    if (p.splits == 1) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<uint32_t*>(p.dk + at + n * 8) =
            pack_bf16x2(dk[n][2 * i] * p.scale, dk[n][2 * i + 1] * p.scale);
        *reinterpret_cast<uint32_t*>(p.dv + at + n * 8) = pack_bf16x2(dv[n][2 * i], dv[n][2 * i + 1]);
      }
    } else {
      const size_t stride = (size_t)p.Nk * p.Hkv * D;
      float* to = p.kv_part + (size_t)split * 2 * stride + at;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        *reinterpret_cast<float2*>(to + n * 8) = make_float2(dk[n][2 * i], dk[n][2 * i + 1]);
        *reinterpret_cast<float2*>(to + stride + n * 8) = make_float2(dv[n][2 * i], dv[n][2 * i + 1]);
      }
    }
  }
}

constexpr int kSumRows = 8, kSumThreads = 256;

// dk = scale x the splits' sums in order, dv likewise without the scale; only rows of segments
template <int D>
__global__ void __launch_bounds__(kSumThreads) rp_dkv_join_kernel(const Params p) {
  int first, klo, khi;
  const int seg = seg_of_tile(p.off_k, p.S, p.Nk, kSumRows, blockIdx.x, first);
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int row0 = klo + ((int)blockIdx.x - first) * kSumRows;
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
        make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
  }
}

static lsrm_status launched() { return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA; }

template <typename K>
static bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 48 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <int D, int NA>
static lsrm_status run_bwd(const Params& p, const BwdPlan& b, cudaStream_t s) {
  lsrm_status st = LSRM_OK;
  const int bins = NA * p.NB;
  if (p.Nq > 0) {
    const size_t bytes = BwdCfg<D, NA>::smem_dq(p.maxd, p.NB);
    if (!allow_smem(rp_dq_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
    rp_dq_kernel<D, NA><<<(unsigned)(b.dq_tiles * p.Hq), kBThreads, bytes, s>>>(p);
    if ((st = launched()) != LSRM_OK) return st;
  }
  rp_table_kernel<<<dim3((unsigned)((bins + 31) / 32), (unsigned)p.Hq), 1024, 0, s>>>(
      p, p.Nq > 0 ? (int)b.dq_tiles : 0, bins);
  if ((st = launched()) != LSRM_OK || p.Nk == 0) return st;
  const size_t bytes = BwdCfg<D, NA>::smem_dkv(p.maxd);
  if (!allow_smem(rp_dkv_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
  rp_dkv_kernel<D, NA><<<(unsigned)(b.kv_tiles * p.Hkv * p.splits), kBThreads, bytes, s>>>(p);
  if ((st = launched()) != LSRM_OK || p.splits == 1) return st;
  rp_dkv_join_kernel<D><<<(unsigned)(p.Nk / kSumRows + p.S), kSumThreads, 0, s>>>(p);
  return launched();
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
