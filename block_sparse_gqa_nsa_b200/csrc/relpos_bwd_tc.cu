// Backward of the attention with a learned relative position bias by buckets on the 5th-generation
// tensor cores: the kernels of long segments (relpos_bwd.cu has the mathematics, the kernels of short
// segments and the joins; relpos_tc.cuh what a thread-per-row layout buys).
//
//   * rp_dq_tc_kernel: a tile of 128 queries of one head, keys in chunks of 64:
//       S = Q K^T, dP = dO V^T (tensor memory) -> P, dS (bf16, tensor memory) -> dQ += dS K, PK += P K, which
//       Delta's correction takes;
//   * rp_dkv_tc_kernel: a tile of 128 keys of one KV head, the queries of its heads in chunks of 64:
//       S^T = K Q^T, dP^T = V dO^T -> P^T, dS^T (bf16, tensor memory) -> dV += P^T dO, dK += dS^T Q, and
//       the table's gradient.
//
// 320 threads: warp 0 brings the streamed operands by TMA and the columns' positions and row constants by
// plain loads, warp 1 issues the MMAs, warps 2-9 do the scores: two threads a row, 32 columns each.  Each
// half of the columns is a pipeline of its own (scores, products, barriers), so that with two CTAs an SM
// four pipelines cover each other's hand-overs between the score warps and the tensor cores (4096 tokens, 32
// heads of 32: dq 365 us, dk/dv 491; before dq had PK, it went 375 -> 338 and dk/dv 573 -> 483 when one pipeline a
// tile was split).  The score warps are the bound: 2.0 to 2.3 warp instructions a clock and SM, the tensor pipe 13 to
// 18%.
// Against the mma.sync kernels, which they replace on long segments, the operands need no shared-memory
// reads by the warps that compute, and runs of columns on one position share look-ups and sums.
//
// Tensor memory (256 columns), in both: at d = 32  S 64 | dP 64 | P 32 | dS 32 | two sums of 32 (PK and dQ, dV and dK),
// at d = 64  S 64 (P over it) | dP 64 (dS over it) | two sums of 64, where each half's P lies over that half's own
// columns and the next scores wait for the products.
#include "relpos_tc.cuh"

namespace lsrm {
namespace rp {

constexpr int kEwThreads = 256;

// A barrier of the eight score warps alone, with the bounded wait of every other (false: gave up)
struct EwBarrier {
  uint64_t* bar;
  volatile int* abort;
  uint32_t* status;
  uint32_t phase;
  __device__ __forceinline__ bool sync() {
    __syncwarp();
    mbar_arrive(bar);
    const bool ok = wait_bar_w(bar, phase & 1, abort, status);
    ++phase;
    return ok;
  }
};

// The bias table of one head by the score warps (index ew = 0..255), as fill_units; vote is a shared word
template <int NA>
__device__ __forceinline__ bool ew_fill(const Params& p, float* lut, int h, int ew, volatile int* vote, EwBarrier& eb,
                                        bool& ok) {
  const int n = 2 * p.maxd + 1;
  if (ew == 0) *vote = 1;
  ok = eb.sync() && ok;  // and every look-up in the old table is over
  bool small = true;
  for (int i = ew; i < n; i += kEwThreads) {
    const int b = checked_bucket(p, i);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const float x = b < 0 ? 0.0f : bf16_to_f32(p.table[((size_t)a * p.NB + b) * p.Hq + h]);
      small = small && (fabsf(x) <= kSmallBias || x == -INFINITY);
      lut[a * n + i] = x;
    }
  }
  if (!small) *vote = 0;
  ok = eb.sync() && ok;
  const bool fold = *vote != 0;
  if (fold) {  // every thread scales the entries that it wrote
    for (int i = ew; i < n; i += kEwThreads)
#pragma unroll
      for (int a = 0; a < NA; ++a) lut[a * n + i] *= kLog2e;
  }
  ok = eb.sync() && ok;
  return fold;
}

// ---- dq -------------------------------------------------------------------------------------------

template <int D>
struct DqTc : TcTile<D> {
  static constexpr int kStages = 3;
  static constexpr bool kAlias = D == 64;
  static constexpr int kColS = 0, kColDp = 64;
  static constexpr int kColP = kAlias ? 0 : 128, kColDs = kAlias ? 64 : 160;
  static constexpr int kHalf = kAlias ? 32 : 16;  // columns from one half's operand to the other's
  static constexpr int kColPk = kAlias ? 128 : 192, kColDq = kColPk + D;
  static_assert(kColDq + D <= 256, "tensor memory");
};
template <int D, int NA>
struct DqTcSmem {
  using C = DqTc<D>;
  uint8_t q[C::kRowsBytes];
  uint8_t o[C::kRowsBytes];  // dO
  uint8_t k[C::kStages][C::kColsBytes];
  uint8_t v[C::kStages][C::kColsBytes];
  int pos[C::kStages][NA][kTcCols];
  ChunkMeta meta[C::kStages];
  uint64_t q_full, kv_full[C::kStages], kv_empty[C::kStages], s_full[2], p_full[2], done[2], drain, ew;
  float rest[2][128], sum[2][128];
  uint32_t tmem_base;
  int abort, vote;
  float lut[1];  // [NA][2 maxd + 1]
  static size_t bytes(int maxd) { return sizeof(DqTcSmem) + (size_t)NA * (2 * maxd + 1) * 4; }
};

template <int D, int NA>
__global__ void __launch_bounds__(kTcThreads, 2)
    rp_dq_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap,
                    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const Params p) {
  using C = DqTc<D>;
  using Smem = DqTcSmem<D, NA>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  if (smem_u32(smem_raw) & 1023) {
    raise_status(p.status, LSRM_ERR_CUDA);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hq, tile = blockIdx.x / p.Hq, hk = h / p.G;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, 128, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + (tile - first) * 128;
  if (tile < first || row0 >= qhi) return;
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int chunks = (khi - klo + kTcCols - 1) / kTcCols, top = 2 * p.maxd;

  if (tid == 0) {
    S.abort = 0;
    mbar_init(&S.q_full, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&S.kv_full[s], 1);
      mbar_init(&S.kv_empty[s], 1);
    }
    for (int hf = 0; hf < 2; ++hf) {
      mbar_init(&S.s_full[hf], 1);
      mbar_init(&S.p_full[hf], kEwThreads / 2);
      mbar_init(&S.done[hf], 1);
    }
    mbar_init(&S.drain, 1);
    mbar_init(&S.ew, kEwThreads);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0 && chunks > 0) {
      mbar_arrive_expect_tx(&S.q_full, 2 * C::kRowsBytes);
      tma_load_3d(S.q, &qmap, &S.q_full, 0, h, row0);
      tma_load_3d(S.o, &omap, &S.q_full, 0, h, row0);
    }
    int issued = 0;
    for (int c = 0; c < chunks; ++c) {
      const int st = c % C::kStages, key = klo + c * kTcCols, n = min(kTcCols, khi - key);
      int x[NA][2];
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i)  // positions past the end repeat the last key's
          x[a][i] = p.pos_k[(size_t)(key + min(lane + 32 * i, n - 1)) * NA + a];
      if (c >= C::kStages && !wait_bar_w(&S.kv_empty[st], ((c / C::kStages) + 1) & 1, abort, p.status)) break;
      note_positions<NA>(x, S.pos[st], S.meta[st], lane, p.status);
      if (n < kTcCols) {
        copy_tail<D>(S.k[st], p.k, key, n, p.Hkv, hk, lane);
        fence_async();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&S.kv_full[st], (n < kTcCols ? 1 : 2) * C::kColsBytes);
        if (n == kTcCols) tma_load_3d(S.k[st], &kmap, &S.kv_full[st], 0, hk, key);
        tma_load_3d(S.v[st], &vmap, &S.kv_full[st], 0, hk, key);
      }
      issued = c + 1;
    }
    if (lane == 0 && *abort) {
      // let the copies already issued land before the CTA's shared memory goes away
      volatile int no_abort = 0;
      if (chunks > 0) wait_bar(&S.q_full, 0, &no_abort, nullptr);
      for (int c = max(0, issued - C::kStages); c < issued; ++c)
        wait_bar(&S.kv_full[c % C::kStages], (c / C::kStages) & 1, &no_abort, nullptr);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0 && chunks > 0) {
      bool ok = wait_bar(&S.q_full, 0, abort, p.status);
      tc_fence_after();
      const uint64_t qdesc = smem_desc(smem_u32(S.q), 16, C::kAtomBytes, C::kLayout);
      const uint64_t odesc = smem_desc(smem_u32(S.o), 16, C::kAtomBytes, C::kLayout);
      const uint64_t kdesc = smem_desc(smem_u32(S.k[0]), 16, C::kAtomBytes, C::kLayout);
      const uint64_t vdesc = smem_desc(smem_u32(S.v[0]), 16, C::kAtomBytes, C::kLayout);
      const uint64_t ksum = smem_desc(smem_u32(S.k[0]), C::kColsBytes, C::kAtomBytes, C::kLayout);
      constexpr uint32_t kStep = C::kColsBytes >> 4, kHalfStep = kStep / 2;
      auto issue_scores = [&](int c, int hf) {
        const uint64_t at = (uint64_t)((c % C::kStages) * kStep + hf * kHalfStep);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + C::kColS + 32 * hf, qdesc + 2 * i, kdesc + at + 2 * i, C::kIdescHalf, i > 0 ? 1u : 0u);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + C::kColDp + 32 * hf, odesc + 2 * i, vdesc + at + 2 * i, C::kIdescHalf, i > 0 ? 1u : 0u);
        mma_commit(&S.s_full[hf]);
      };
      auto issue_sums = [&](int c, int hf) {
        const uint64_t at = (uint64_t)((c % C::kStages) * kStep + hf * kHalfStep);
        const uint32_t first_add = c == 0 && hf == 0 ? 0u : 1u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_ts(tmem + C::kColPk, tmem + C::kColP + hf * C::kHalf + i * 8, ksum + at + i * (16 * C::kRowBytes >> 4),
                 C::kIdescSum, i == 0 ? first_add : 1u);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_ts(tmem + C::kColDq, tmem + C::kColDs + hf * C::kHalf + i * 8, ksum + at + i * (16 * C::kRowBytes >> 4),
                 C::kIdescSum, i == 0 ? first_add : 1u);
        mma_commit(&S.done[hf]);
      };
      for (int c = 0; ok && c < chunks; ++c) {
        if (!wait_bar(&S.kv_full[c % C::kStages], (c / C::kStages) & 1, abort, p.status)) { ok = false; break; }
        for (int hf = 0; hf < 2; ++hf) {
          if (c > 0 && !wait_bar(&S.p_full[hf], (c - 1) & 1, abort, p.status)) { ok = false; break; }
          tc_fence_after();
          if (!C::kAlias) issue_scores(c, hf);  // S and dP were released with dS(c - 1)
          if (c > 0) issue_sums(c - 1, hf);
        }
        if (!ok) break;
        if (c > 0) mma_commit(&S.kv_empty[(c - 1) % C::kStages]);
        if (C::kAlias) {
          for (int hf = 0; hf < 2; ++hf) {
            // the next scores overwrite the operands of the products, so those have to be done
            if (c > 0 && !wait_bar(&S.done[hf], (c - 1) & 1, abort, p.status)) { ok = false; break; }
            tc_fence_after();
            issue_scores(c, hf);
          }
        }
      }
      for (int hf = 0; ok && hf < 2; ++hf) {
        if (!wait_bar(&S.p_full[hf], (chunks - 1) & 1, abort, p.status)) { ok = false; break; }
        tc_fence_after();
        issue_sums(chunks - 1, hf);
      }
      // every MMA issued so far must finish before the CTA can release tensor and shared memory
      mma_commit(&S.drain);
      volatile int no_abort = 0;
      wait_bar(&S.drain, 0, &no_abort, nullptr);
    }
  } else {
    // ---------------- scores: two threads a row ----------------
    const int ew = tid - 64, half = ew >> 7, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16);
    const int row = row0 + r;
    const bool valid = row < qhi;
    const size_t at = (size_t)(valid ? row : row0) * p.Hq + h;
    int rowc[NA], q_lo[NA], q_hi[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int x = p.pos_q[(size_t)min(row, qhi - 1) * NA + a];
      rowc[a] = p.maxd - x;
      q_lo[a] = __reduce_min_sync(0xffffffffu, x);
      q_hi[a] = __reduce_max_sync(0xffffffffu, x);
      if (q_lo[a] < -kPosLimit || q_hi[a] > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
    }
    EwBarrier eb{&S.ew, abort, p.status, 0};
    bool ok = true;
    const bool small = ew_fill<NA>(p, S.lut, h, ew, &S.vote, eb, ok);
    const float mul = small ? p.scale * kLog2e : p.scale;
    const float lse = row_lse(valid ? p.lse_in[at] : INFINITY), rconst = row_const(lse, small);
    float delta = 0.0f, rest = 0.0f, sum = 0.0f;
    if (valid) {
      const uint4* a = reinterpret_cast<const uint4*>(p.dout + at * D);
      const uint4* b = reinterpret_cast<const uint4*>(p.o_in + at * D);
#pragma unroll 2
      for (int i = 0; i < D / 8; ++i) {
        const uint4 u = a[i], w = b[i];
        const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          delta = fmaf(bf16_to_f32((uint16_t)us[e]), bf16_to_f32((uint16_t)ws[e]), delta);
          delta = fmaf(__uint_as_float(us[e] & 0xffff0000u), __uint_as_float(ws[e] & 0xffff0000u), delta);
        }
      }
    }
    __syncwarp();
    const bool exact = !small || __any_sync(0xffffffffu, is_huge(lse));

    ChunkBias<NA> cb;
    for (int c = 0; ok && c < chunks; ++c) {
      const int st = c % C::kStages, left = khi - klo - c * kTcCols;
      if (!wait_bar_w(&S.kv_full[st], (c / C::kStages) & 1, abort, p.status) ||
          !wait_bar_w(&S.s_full[half], c & 1, abort, p.status) ||
          (!C::kAlias && c > 0 && !wait_bar_w(&S.done[half], (c - 1) & 1, abort, p.status))) {  // P and dS are free
        ok = false;
        break;
      }
      tc_fence_after();
      cb.set(S.meta[st], q_lo, q_hi, p.maxd, S.lut, top);
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {
        const int col = half * 32 + g * 16;
        uint32_t s[16], d[16];
        tmem_ld16(tbase + C::kColS + col, s);
        tmem_ld16(tbase + C::kColDp + col, d);
        tmem_wait16(s);
        tmem_wait16(d);
        float x[16];
        if (!exact) {  // the row's constant with the bias
          const float b = cb.row16(cb.ub - rconst, S.pos[st], 2 * half + g, rowc, S.lut, top);
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            ffma2(x[e], x[e + 1], __uint_as_float(s[e]), __uint_as_float(s[e + 1]), mul, b);
          if (!cb.flat(2 * half + g)) cb.add16(x, S.pos[st], 2 * half + g, rowc, S.lut, top);
        } else {
          keep_branch();
          cb.exact16(x, s, mul, S.pos[st], 2 * half + g, rowc, S.lut, top);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] -= rconst;
            if (!small) x[e] *= kLog2e;
          }
        }
        if (left < col + 16) {  // no key: P = 0, and dP may be anything
          keep_branch();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (col + e >= left) x[e] = -INFINITY, d[e] = 0;
        }
        float s0 = 0.0f, s1 = 0.0f, l0 = 0.0f, l1 = 0.0f;
        uint32_t pp[8], pd[8];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float p0 = ex2(x[e]), p1 = ex2(x[e + 1]);
          float d0 = __uint_as_float(d[e]), d1 = __uint_as_float(d[e + 1]);
          fadd2_acc(d0, d1, -delta, -delta);
          fmul2(d0, d1, d0, d1, p0, p1);
          fadd2_acc(s0, s1, d0, d1);
          fadd2_acc(l0, l1, p0, p1);
          pp[e / 2] = pack2(p0, p1);
          pd[e / 2] = pack2(d0, d1);
        }
        rest += s0 + s1;
        sum += l0 + l1;
        tmem_st8(tbase + C::kColP + half * C::kHalf + g * 8, pp);
        tmem_st8(tbase + C::kColDs + half * C::kHalf + g * 8, pd);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&S.p_full[half]);
    }
    if (ok && chunks > 0)
      ok = wait_bar_w(&S.done[0], (chunks - 1) & 1, abort, p.status) &&
           wait_bar_w(&S.done[1], (chunks - 1) & 1, abort, p.status);
    tc_fence_after();
    S.rest[half][r] = rest;
    S.sum[half][r] = sum;
    ok = eb.sync() && ok;
    const float l = S.sum[0][r] + S.sum[1][r], inv = valid ? row_inverse(l, rconst, p.status) : 0.0f;
    const float more = (S.rest[0][r] + S.rest[1][r]) * inv, f = inv * p.scale;  // more: Delta less the saved out's
    if (half == 0 && valid) {
      const float corr = row_corr(l);
      p.delta[at] = delta + more;
      p.lse2[at] = row_lse2(rconst, small, corr);
      p.corr[at] = corr;
    }
    // each thread half of the row's dq
#pragma unroll 1
    for (int i = 0; i < D / 32; ++i) {
      uint32_t o[16], k[16];
      const int col = half * (D / 2) + i * 16;
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = k[e] = 0;
      if (ok && chunks > 0) {
        tmem_ld16(tbase + C::kColDq + col, o);
        tmem_wait16(o);
        tmem_ld16(tbase + C::kColPk + col, k);
        tmem_wait16(k);
      }
      if (!valid) continue;
      float x[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = fmaf(-more, __uint_as_float(k[e]), __uint_as_float(o[e])) * f;
      uint32_t u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = pack2(x[2 * e], x[2 * e + 1]);
      uint4* dst = reinterpret_cast<uint4*>(p.dq + at * D + col);
      dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
      dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---- dk, dv and the table's gradient ---------------------------------------------------------------

// The table's sums stand in columns that one thread at a time adds to: a thread's own, or, with several
// axes, one column per axis for the two threads of a key, who work on different axes at any time and change
// over in turns.  That halves the sums (32 buckets, two axes: 68 -> 34 KB) and lets two CTAs share an SM,
// which the work behind every score's look-ups needs: dk, dv and table of six frames of 1370 tokens (16 heads
// of 64, two axes) 698 -> 552 us, 1024 tokens of three axes (32 heads of 32, whole backward) 226 -> 192 us.
// Where two CTAs do not fit in any case, a CTA has the registers of both, own columns and a third stage
// (64 buckets, whole backward: 987 us; turns without company: 1125 us).
template <int D, int NA, int CTAS>
struct DkvTc : TcTile<D> {
  static constexpr int kStages = D == 32 || CTAS == 1 ? 3 : 2;
  static constexpr bool kTurns = NA > 1 && CTAS == 2;
  static constexpr int kSums = kTurns ? kEwThreads / 2 : kEwThreads;
  static constexpr bool kAlias = D == 64;
  static constexpr int kColS = 0, kColDp = 64;
  static constexpr int kColP = kAlias ? 0 : 128, kColDs = kAlias ? 64 : 160;
  static constexpr int kHalf = kAlias ? 32 : 16;  // columns from one half's operand to the other's
  static constexpr int kColDv = kAlias ? 128 : 192, kColDk = kColDv + D;
  static_assert(kColDk + D <= 256, "tensor memory");
};
template <int D, int NA, int CTAS>
struct DkvTcSmem {
  using C = DkvTc<D, NA, CTAS>;
  uint8_t k[C::kRowsBytes];
  uint8_t v[C::kRowsBytes];
  uint8_t q[C::kStages][C::kColsBytes];
  uint8_t o[C::kStages][C::kColsBytes];  // dO
  int pos[C::kStages][NA][kTcCols];
  float nlse[C::kStages][kTcCols], ndelta[C::kStages][kTcCols];  // negated: packed adds have no signs
  ChunkMeta meta[C::kStages];
  uint64_t k_full, q_full[C::kStages], q_empty[C::kStages], s_full[2], p_full[2], done[2], drain, ew, turn[4];
  uint32_t tmem_base;
  int abort, vote, pad;
  int huge[C::kStages][2];  // whether a half of the columns has a row of huge |LSE|
  // behind it: table fp32 [NA][2 maxd + 1], the buckets' byte offsets int32 [2 maxd + 1], and the
  // columns of sums fp32 [NA][NB and one for ids out of range][kSums]
  static size_t bytes(int maxd, int nb) {
    return sizeof(DkvTcSmem) + (size_t)(NA + 1) * (2 * maxd + 1) * 4 + (size_t)NA * (nb + 1) * C::kSums * 4;
  }
};

template <int D, int NA, int CTAS>
__global__ void __launch_bounds__(kTcThreads, CTAS)
    rp_dkv_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap,
                     const Params p) {
  using C = DkvTc<D, NA, CTAS>;
  using Smem = DkvTcSmem<D, NA, CTAS>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  if (smem_u32(smem_raw) & 1023) {
    raise_status(p.status, LSRM_ERR_CUDA);
    return;
  }
  const int top = 2 * p.maxd, bins = NA * p.NB;
  float* lut = reinterpret_cast<float*>(smem_raw + sizeof(Smem));
  int* boff = reinterpret_cast<int*>(lut + NA * (top + 1));
  float* hist = reinterpret_cast<float*>(boff + top + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_dependents();
  int unit = blockIdx.x;
  const int split = unit % p.splits;
  unit /= p.splits;
  const int hk = unit % p.Hkv, tile = unit / p.Hkv;
  int first, qlo = 0, qhi = 0, klo, khi;
  const int seg = seg_of_tile(p.off_k, p.S, p.Nk, 128, tile, first);
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int row0 = klo + (tile - first) * 128;
  const bool empty = tile < first || row0 >= khi;
  if (!empty) seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int chunks = (qhi - qlo + kTcCols - 1) / kTcCols;
  int h0, h1, c0, c1, part;
  split_range(p, split, chunks, h0, h1, c0, c1, part);
  const int parts = p.splits > p.G ? p.splits / p.G : 1;
  float* tab_part = p.tab_part + (((size_t)tile * parts + part) * p.Hq + hk * p.G) * bins;  // + head * bins
  const int nc = c1 - c0, steps = (h1 - h0) * nc;
  if (empty || steps == 0)  // no pair: the table's sums are 0
    for (int i = h0 * bins + tid; i < h1 * bins; i += kTcThreads) tab_part[i] = 0.0f;
  if (empty) return;

  if (tid == 0) {
    S.abort = 0;
    mbar_init(&S.k_full, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&S.q_full[s], 1);
      mbar_init(&S.q_empty[s], 1);
    }
    for (int hf = 0; hf < 2; ++hf) {
      mbar_init(&S.s_full[hf], 1);
      mbar_init(&S.p_full[hf], kEwThreads / 2);
      mbar_init(&S.done[hf], 1);
    }
    mbar_init(&S.drain, 1);
    mbar_init(&S.ew, kEwThreads);
    for (int i = 0; i < 4; ++i) mbar_init(&S.turn[i], 2);
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0 && steps > 0) {
      mbar_arrive_expect_tx(&S.k_full, 2 * C::kRowsBytes);
      tma_load_3d(S.k, &kmap, &S.k_full, 0, hk, row0);
      tma_load_3d(S.v, &vmap, &S.k_full, 0, hk, row0);
    }
    int issued = 0;
    for (int it = 0; it < steps; ++it) {
      const int st = it % C::kStages, h = hk * p.G + h0 + it / nc, q0 = qlo + (c0 + it % nc) * kTcCols;
      const int n = min(kTcCols, qhi - q0);
      int x[NA][2];
      float l[2], dl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const size_t q = q0 + min(lane + 32 * i, n - 1);  // past the end the last query's
#pragma unroll
        for (int a = 0; a < NA; ++a) x[a][i] = -p.pos_q[q * NA + a];  // negated, as the keys' below
        l[i] = lane + 32 * i < n ? p.lse2[q * p.Hq + h] : INFINITY;  // no query: P = 0
        dl[i] = p.delta[q * p.Hq + h];
      }
      if (it >= C::kStages && !wait_bar_w(&S.q_empty[st], ((it / C::kStages) + 1) & 1, abort, p.status)) break;
      note_positions<NA>(x, S.pos[st], S.meta[st], lane, p.status);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        S.nlse[st][lane + 32 * i] = -l[i];
        S.ndelta[st][lane + 32 * i] = -dl[i];
        const bool huge = __any_sync(0xffffffffu, is_huge(l[i]));
        if (lane == 0) S.huge[st][i] = huge;
      }
      if (n < kTcCols) {
        copy_tail<D>(S.q[st], p.q, q0, n, p.Hq, h, lane);
        copy_tail<D>(S.o[st], p.dout, q0, n, p.Hq, h, lane);
        fence_async();
      }
      __syncwarp();
      if (lane == 0) {
        if (n == kTcCols) {
          mbar_arrive_expect_tx(&S.q_full[st], 2 * C::kColsBytes);
          tma_load_3d(S.q[st], &qmap, &S.q_full[st], 0, h, q0);
          tma_load_3d(S.o[st], &omap, &S.q_full[st], 0, h, q0);
        } else {
          mbar_arrive(&S.q_full[st]);
        }
      }
      issued = it + 1;
    }
    if (lane == 0 && *abort) {
      volatile int no_abort = 0;
      if (steps > 0) wait_bar(&S.k_full, 0, &no_abort, nullptr);
      for (int c = max(0, issued - C::kStages); c < issued; ++c)
        wait_bar(&S.q_full[c % C::kStages], (c / C::kStages) & 1, &no_abort, nullptr);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (lane == 0 && steps > 0) {
      bool ok = wait_bar(&S.k_full, 0, abort, p.status);
      tc_fence_after();
      const uint64_t kdesc = smem_desc(smem_u32(S.k), 16, C::kAtomBytes, C::kLayout);
      const uint64_t vdesc = smem_desc(smem_u32(S.v), 16, C::kAtomBytes, C::kLayout);
      const uint64_t qdesc = smem_desc(smem_u32(S.q[0]), 16, C::kAtomBytes, C::kLayout);
      const uint64_t odesc = smem_desc(smem_u32(S.o[0]), 16, C::kAtomBytes, C::kLayout);
      const uint64_t qsum = smem_desc(smem_u32(S.q[0]), C::kColsBytes, C::kAtomBytes, C::kLayout);
      const uint64_t osum = smem_desc(smem_u32(S.o[0]), C::kColsBytes, C::kAtomBytes, C::kLayout);
      constexpr uint32_t kStep = C::kColsBytes >> 4, kHalfStep = kStep / 2;
      auto issue_scores = [&](int it, int hf) {
        const uint64_t at = (uint64_t)((it % C::kStages) * kStep + hf * kHalfStep);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + C::kColS + 32 * hf, kdesc + 2 * i, qdesc + at + 2 * i, C::kIdescHalf, i > 0 ? 1u : 0u);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(tmem + C::kColDp + 32 * hf, vdesc + 2 * i, odesc + at + 2 * i, C::kIdescHalf, i > 0 ? 1u : 0u);
        mma_commit(&S.s_full[hf]);
      };
      auto issue_sums = [&](int it, int hf) {
        const uint64_t at = (uint64_t)((it % C::kStages) * kStep + hf * kHalfStep);
        const uint32_t first_add = it == 0 && hf == 0 ? 0u : 1u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_ts(tmem + C::kColDv, tmem + C::kColP + hf * C::kHalf + i * 8, osum + at + i * (16 * C::kRowBytes >> 4),
                 C::kIdescSum, i == 0 ? first_add : 1u);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_ts(tmem + C::kColDk, tmem + C::kColDs + hf * C::kHalf + i * 8, qsum + at + i * (16 * C::kRowBytes >> 4),
                 C::kIdescSum, i == 0 ? first_add : 1u);
        mma_commit(&S.done[hf]);
      };
      for (int it = 0; ok && it < steps; ++it) {
        if (!wait_bar(&S.q_full[it % C::kStages], (it / C::kStages) & 1, abort, p.status)) { ok = false; break; }
        for (int hf = 0; hf < 2; ++hf) {
          if (it > 0 && !wait_bar(&S.p_full[hf], (it - 1) & 1, abort, p.status)) { ok = false; break; }
          tc_fence_after();
          if (!C::kAlias) issue_scores(it, hf);
          if (it > 0) issue_sums(it - 1, hf);
        }
        if (!ok) break;
        if (it > 0) mma_commit(&S.q_empty[(it - 1) % C::kStages]);
        if (C::kAlias) {
          for (int hf = 0; hf < 2; ++hf) {
            // the next scores overwrite the operands of the products, so those have to be done
            if (it > 0 && !wait_bar(&S.done[hf], (it - 1) & 1, abort, p.status)) { ok = false; break; }
            tc_fence_after();
            issue_scores(it, hf);
          }
        }
      }
      for (int hf = 0; ok && hf < 2; ++hf) {
        if (!wait_bar(&S.p_full[hf], (steps - 1) & 1, abort, p.status)) { ok = false; break; }
        tc_fence_after();
        issue_sums(steps - 1, hf);
      }
      mma_commit(&S.drain);
      volatile int no_abort = 0;
      wait_bar(&S.drain, 0, &no_abort, nullptr);
    }
  } else {
    // ---------------- scores: two threads a key ----------------
    const int ew = tid - 64, half = ew >> 7, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16);
    const int row = row0 + r;
    const bool valid = row < khi;
    int rowc[NA], k_lo[NA], k_hi[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      // delta = (- pos_q) - (- pos_k): with both negated, columns less rows as in the other kernels
      const int x = -p.pos_k[(size_t)min(row, khi - 1) * NA + a];
      rowc[a] = p.maxd - x;
      k_lo[a] = __reduce_min_sync(0xffffffffu, x);
      k_hi[a] = __reduce_max_sync(0xffffffffu, x);
    }
    for (int i = ew; i < top + 1; i += kEwThreads) {
      const int b = p.bucket_of[i];
      boff[i] = (b < 0 || b >= p.NB ? p.NB : b) * C::kSums * 4;
    }
    const int axis_bytes = (p.NB + 1) * C::kSums * 4;
    for (int i = ew; i < NA * (p.NB + 1) * C::kSums; i += kEwThreads) hist[i] = 0.0f;
    char* mine = reinterpret_cast<char*>(hist + (C::kTurns ? r : ew));
    // the running sum of chunks on one distance, and its bucket's offset
    float run[NA];
    int run_b[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) run[a] = 0.0f, run_b[a] = p.NB * C::kSums * 4;

    EwBarrier eb{&S.ew, abort, p.status, 0};
    bool ok = true, small = false;
    float mul = 0.0f;
    ChunkBias<NA> cb;
    uint32_t turn = 0;
    // a turn: the two warps that share keys have both come here
    auto swap = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.turn[quarter]);
      ok = wait_bar_w(&S.turn[quarter], turn & 1, abort, p.status) && ok;
      ++turn;
    };
    for (int it = 0; ok && it < steps; ++it) {
      const int st = it % C::kStages, cc = it % nc, head = h0 + it / nc;
      if (cc == 0) {
        small = ew_fill<NA>(p, lut, hk * p.G + head, ew, &S.vote, eb, ok);
        mul = small ? p.scale * kLog2e : p.scale;
      }
      if (!wait_bar_w(&S.q_full[st], (it / C::kStages) & 1, abort, p.status) ||
          !wait_bar_w(&S.s_full[half], it & 1, abort, p.status) ||
          (!C::kAlias && it > 0 && !wait_bar_w(&S.done[half], (it - 1) & 1, abort, p.status))) {  // P and dS are free
        ok = false;
        break;
      }
      tc_fence_after();
      cb.set(S.meta[st], k_lo, k_hi, p.maxd, lut, top);
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {
        const int col = half * 32 + g * 16;
        uint32_t s[16], d[16];
        tmem_ld16(tbase + C::kColS + col, s);
        tmem_ld16(tbase + C::kColDp + col, d);
        tmem_wait16(s);
        tmem_wait16(d);
        const float4* ls = reinterpret_cast<const float4*>(&S.nlse[st][col]);
        const float4* ds = reinterpret_cast<const float4*>(&S.ndelta[st][col]);
        float x[16];
        if (small && !S.huge[st][half]) {
          const float b = cb.row16(cb.ub, S.pos[st], 2 * half + g, rowc, lut, top);
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            float4 l = ls[f];
            fadd2_acc(l.x, l.y, b, b);
            fadd2_acc(l.z, l.w, b, b);
            ffma2v(x[4 * f], x[4 * f + 1], __uint_as_float(s[4 * f]), __uint_as_float(s[4 * f + 1]), mul, l.x, l.y);
            ffma2v(x[4 * f + 2], x[4 * f + 3], __uint_as_float(s[4 * f + 2]), __uint_as_float(s[4 * f + 3]), mul, l.z,
                   l.w);
          }
          if (!cb.flat(2 * half + g)) cb.add16(x, S.pos[st], 2 * half + g, rowc, lut, top);
        } else {
          // the row's constant and the correction one after the other: together they would be rounded to the
          // former's spacing
          keep_branch();
          cb.exact16(x, s, mul, S.pos[st], 2 * half + g, rowc, lut, top);
          const int q = qlo + (c0 + cc) * kTcCols + col;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const size_t at = (size_t)min(q + e, qhi - 1) * p.Hq + hk * p.G + head;
            x[e] -= row_const(q + e < qhi ? row_lse(p.lse_in[at]) : INFINITY, small);
            x[e] = small ? x[e] - p.corr[at] : fmaf(x[e], kLog2e, -p.corr[at]);
          }
        }
        uint32_t pp[8], pd[8];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const float4 dl = ds[f];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int i = 4 * f + e;
            const float p0 = ex2(x[i]), p1 = ex2(x[i + 1]);
            float d0 = __uint_as_float(d[i]), d1 = __uint_as_float(d[i + 1]);
            fadd2_acc(d0, d1, e == 0 ? dl.x : dl.z, e == 0 ? dl.y : dl.w);
            fmul2(x[i], x[i + 1], d0, d1, p0, p1);
            pp[i / 2] = pack2(p0, p1);
            pd[i / 2] = pack2(x[i], x[i + 1]);
          }
        }
        tmem_st8(tbase + C::kColP + half * C::kHalf + g * 8, pp);
        tmem_st8(tbase + C::kColDs + half * C::kHalf + g * 8, pd);
        if (!valid) {  // a row past the segment's last key has no pairs (its operands may be anything)
          keep_branch();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.0f;
        }
        __syncwarp();
        // the table's gradient.  In turns: the halves are on axes ph and ph + 1, forwards in a run of
        // columns and back in the next, so that a run begins where the one before it ended.
#pragma unroll 1
        for (int ph = 0; ph < (C::kTurns ? NA : 1); ++ph) {
          if (ph > 0) swap();
          const int place = (g == 0 ? ph : NA - 1 - ph) + half, axis = place < NA ? place : place - NA;
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            if (C::kTurns && a != axis) continue;
            char* to = mine + a * axis_bytes;
            const int4* xs = reinterpret_cast<const int4*>(&S.pos[st][a][col]);
            const int md = cb.mode(a, 2 * half + g);
            if (md <= kLane) {
              float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
              for (int e = 0; e < 16; e += 2) fadd2_acc(s0, s1, x[e], x[e + 1]);
              const int b = boff[md == kOne ? cb.one[a] : clamp_index(xs[0].x, rowc[a], top)];
              if (b != run_b[a]) {
                *reinterpret_cast<float*>(to + run_b[a]) += run[a];
                run[a] = 0.0f;
                run_b[a] = b;
              }
              run[a] += s0 + s1;
            } else if (md == kFour) {
#pragma unroll
              for (int f = 0; f < 4; f += 2)
                add_two(to, boff[clamp_index(xs[f].x, rowc[a], top)],
                           (x[4 * f] + x[4 * f + 1]) + (x[4 * f + 2] + x[4 * f + 3]),
                           boff[clamp_index(xs[f + 1].x, rowc[a], top)],
                           (x[4 * f + 4] + x[4 * f + 5]) + (x[4 * f + 6] + x[4 * f + 7]));
            } else if (kHasTurn<NA> && md == kTurn) {
              const int4 u = xs[0];
              add_two(to, boff[clamp_index(u.x, rowc[a], top)], (x[0] + x[4]) + (x[8] + x[12]),
                         boff[clamp_index(u.y, rowc[a], top)], (x[1] + x[5]) + (x[9] + x[13]));
              add_two(to, boff[clamp_index(u.z, rowc[a], top)], (x[2] + x[6]) + (x[10] + x[14]),
                         boff[clamp_index(u.w, rowc[a], top)], (x[3] + x[7]) + (x[11] + x[15]));
            } else {
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const int4 u = xs[f];
                add_two(to, boff[clamp_index(u.x, rowc[a], top)], x[4 * f], boff[clamp_index(u.y, rowc[a], top)],
                           x[4 * f + 1]);
                add_two(to, boff[clamp_index(u.z, rowc[a], top)], x[4 * f + 2],
                           boff[clamp_index(u.w, rowc[a], top)], x[4 * f + 3]);
              }
            }
          }
        }
        __syncwarp();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&S.p_full[half]);
      if (cc == nc - 1) {
        // the head's sums of the CTA's threads to global memory, and the columns back to 0
#pragma unroll
        for (int turns = 0; turns < (C::kTurns ? 2 : 1); ++turns) {
          if (C::kTurns) ok = eb.sync() && ok;
          if (C::kTurns && turns != half) continue;
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            *reinterpret_cast<float*>(mine + a * axis_bytes + run_b[a]) += run[a];
            run[a] = 0.0f;
          }
        }
        ok = eb.sync() && ok;
        flush_sums<C::kSums, kEwThreads>(hist, bins, p.NB, ew, tab_part + head * bins);
        ok = eb.sync() && ok;
      }
    }
    if (ok && steps > 0)
      ok = wait_bar_w(&S.done[0], (steps - 1) & 1, abort, p.status) &&
           wait_bar_w(&S.done[1], (steps - 1) & 1, abort, p.status);
    tc_fence_after();
    // one half writes dV, the other dK
    const size_t at = ((size_t)(valid ? row : row0) * p.Hkv + hk) * D;
    const size_t stride = (size_t)p.Nk * p.Hkv * D;
    const float f = half == 0 ? 1.0f : p.scale;
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {
      uint32_t o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = 0;
      if (ok && steps > 0) {
        tmem_ld16(tbase + (half == 0 ? C::kColDv : C::kColDk) + 16 * i, o);
        tmem_wait16(o);
      }
      if (!valid) continue;
      if (p.splits == 1) {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = pack2(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
        uint4* dst = reinterpret_cast<uint4*>((half == 0 ? p.dv : p.dk) + at + 16 * i);
        dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
        dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
      } else {
        float* part = p.kv_part + ((size_t)split * 2 + (half == 0 ? 1 : 0)) * stride;
        uint4* dst = reinterpret_cast<uint4*>(part + at + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ---- launch -----------------------------------------------------------------------------------------

// a map of rows x heads boxes; a tensor without tokens is never read, but a map needs an address
static bool map_of(CUtensorMap* m, const uint16_t* base, const uint16_t* other, int D, int heads, int n, int box) {
  return make_map(m, n > 0 ? base : other, D, heads, n > 0 ? n : 1, 1, box);
}

template <int D, int NA, int CTAS>
static lsrm_status run_dkv_tc(const Params& p, const BwdPlan& b, const CUtensorMap& k128, const CUtensorMap& v128,
                              const CUtensorMap& q64, const CUtensorMap& o64, cudaStream_t s) {
  const size_t bytes = DkvTcSmem<D, NA, CTAS>::bytes(p.maxd, p.NB);
  auto* kernel = rp_dkv_tc_kernel<D, NA, CTAS>;
  if (!allow_smem(kernel, bytes)) return LSRM_ERR_CUDA;
  kernel<<<(unsigned)(b.kv_tiles * p.Hkv * p.splits), kTcThreads, bytes, s>>>(k128, v128, q64, o64, p);
  return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

template <int D, int NA>
static lsrm_status run_bwd_tc(const Params& p, const BwdPlan& b, cudaStream_t s) {
  CUtensorMap q128, o128, k64, v64, k128, v128, q64, o64;
  if (!map_of(&q128, p.q, p.k, D, p.Hq, p.Nq, 128) || !map_of(&o128, p.dout, p.k, D, p.Hq, p.Nq, 128) ||
      !map_of(&q64, p.q, p.k, D, p.Hq, p.Nq, 64) || !map_of(&o64, p.dout, p.k, D, p.Hq, p.Nq, 64) ||
      !map_of(&k128, p.k, p.q, D, p.Hkv, p.Nk, 128) || !map_of(&v128, p.v, p.q, D, p.Hkv, p.Nk, 128) ||
      !map_of(&k64, p.k, p.q, D, p.Hkv, p.Nk, 64) || !map_of(&v64, p.v, p.q, D, p.Hkv, p.Nk, 64))
    return LSRM_ERR_CUDA;
  if (p.Nq > 0) {
    const size_t bytes = DqTcSmem<D, NA>::bytes(p.maxd);
    if (!allow_smem(rp_dq_tc_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
    rp_dq_tc_kernel<D, NA><<<(unsigned)(b.dq_tiles * p.Hq), kTcThreads, bytes, s>>>(q128, o128, k64, v64, p);
    if (cudaGetLastError() != cudaSuccess) return LSRM_ERR_CUDA;
  }
  if (p.Nk > 0)
    return b.tc == 2 ? run_dkv_tc<D, NA, 2>(p, b, k128, v128, q64, o64, s)
                     : run_dkv_tc<D, NA, 1>(p, b, k128, v128, q64, o64, s);
  return LSRM_OK;
}

lsrm_status launch_bwd_tc(const Params& p, int D, int NA, const BwdPlan& b, cudaStream_t s) {
  if (D == 32)
    return NA == 1 ? run_bwd_tc<32, 1>(p, b, s) : NA == 2 ? run_bwd_tc<32, 2>(p, b, s) : run_bwd_tc<32, 3>(p, b, s);
  return NA == 1 ? run_bwd_tc<64, 1>(p, b, s) : NA == 2 ? run_bwd_tc<64, 2>(p, b, s) : run_bwd_tc<64, 3>(p, b, s);
}
template <int D, int NA>
static int dkv_fit(int maxd, int nb) {
  if (2 * (DkvTcSmem<D, NA, 2>::bytes(maxd, nb) + 1024) <= 228 * 1024) return 2;
  return DkvTcSmem<D, NA, 1>::bytes(maxd, nb) <= 227 * 1024 ? 1 : 0;
}
int bwd_tc_ctas(int D, int NA, int maxd, int nb) {
  if (D == 32)
    return NA == 1 ? dkv_fit<32, 1>(maxd, nb) : NA == 2 ? dkv_fit<32, 2>(maxd, nb) : dkv_fit<32, 3>(maxd, nb);
  return NA == 1 ? dkv_fit<64, 1>(maxd, nb) : NA == 2 ? dkv_fit<64, 2>(maxd, nb) : dkv_fit<64, 3>(maxd, nb);
}

}  // namespace rp
}  // namespace lsrm
