// Short segments (blocks of a brick or tile of tokens) of the attention with a learned relative position
// bias: forward and dq.  relpos.cuh has the formulas, relpos_bwd.cu the backward's mathematics.
//
// A segment of some tens of tokens is a few score tiles a head, and a CTA of its own for each head spends
// its time on dependent reads: the segment's number, its bounds, the bias table, the operands.  Here one
// CTA takes 64 queries and up to 16 heads of a KV group: the segment is looked up once, K, V and the
// positions are brought to shared memory once, the bias tables of all its heads are filled side by side,
// and the warps walk the (head, 16 queries) units, each fetching the next unit's operands while it works on
// its own.  Longer segments stream their keys in blocks of 64, again for each round of units.
// 256 ragged blocks of up to 64 tokens, 32 heads of 32, three axes: forward 71 us, dq 102; a CTA a head took 85
// and 146.  Bound by instructions (2.1 and 2.0 a clock and SM), most of them around a score: the exponential,
// three look-ups, the tile's edges.
#include "relpos.cuh"

namespace lsrm {
namespace rp {

constexpr int kShWarps = 8, kShThreads = 32 * kShWarps, kShKeys = 64;
constexpr float kShSlack = 8.0f;

template <int D, int NA>
struct ShCfg {
  static constexpr int kTile = kShKeys * D / 8;  // 16-byte pieces of a K or V block
  static constexpr size_t kRing = 2 * ((size_t)2 * kTile * 16 + kShKeys * NA * 4);
  static constexpr int kUnit = 16 * D / 8;  // pieces of 16 rows
  static constexpr size_t kUnits = (size_t)kShWarps * 3 * kUnit * 16;  // dq: the next queries, dO and out of a warp
  static constexpr size_t kFlags = kShWarps * 4;  // a warp's heads with large tables
  static size_t smem(int maxd, int heads, bool dq) {
    return kRing + (dq ? kUnits : 0) + kFlags + (size_t)heads * NA * (2 * maxd + 1) * 4;
  }
};

// the CTA's place: a tile of 64 queries of a segment, heads h0 .. h0 + nh - 1 of KV head hk
struct ShPlace {
  int qlo, qhi, klo, khi, row0, hk, h0, nh;
  bool live;
};
__device__ __forceinline__ ShPlace sh_place(const Params& p) {
  ShPlace s;
  const int GH = min(p.G, kShHeads), hgroups = (p.G + GH - 1) / GH;
  int unit = blockIdx.x;
  const int hg = unit % hgroups;
  unit /= hgroups;
  s.hk = unit % p.Hkv;
  const int tile = unit / p.Hkv;
  int first;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, 64, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, s.qlo, s.qhi, p.status);
  seg_bounds(p.off_k, seg, p.Nk, s.klo, s.khi, p.status);
  s.row0 = s.qlo + (tile - first) * 64;
  s.live = tile >= first && s.row0 < s.qhi;
  s.h0 = s.hk * p.G + hg * GH;
  s.nh = min(GH, p.G - hg * GH);
  return s;
}

// the bias tables of nh heads [head][axis][2 maxd + 1], each in its own units as fill_units has them (the key pass
// takes the heads one by one, and has to come to the same scores).  Returns the heads with large tables, which the warps
// collect in the words in front of the tables.
template <int NA>
__device__ __forceinline__ uint32_t sh_fill(const Params& p, float* lut, int h0, int nh, int tid) {
  const int n = 2 * p.maxd + 1;
  uint32_t* words = reinterpret_cast<uint32_t*>(lut) - kShWarps;
  uint32_t large = 0;
  for (int i = tid; i < n * nh; i += kShThreads) {
    const int d = i / nh, hh = i % nh;
    const int b = checked_bucket(p, d);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const float x = b < 0 ? 0.0f : bf16_to_f32(p.table[((size_t)a * p.NB + b) * p.Hq + h0 + hh]);
      if (!(fabsf(x) <= kSmallBias || x == -INFINITY)) large |= 1u << hh;
      lut[(hh * NA + a) * n + d] = x;
    }
  }
  large = __reduce_or_sync(0xffffffffu, large);
  if ((tid & 31) == 0) words[tid >> 5] = large;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kShWarps; ++w) large |= words[w];
  for (int i = tid; i < n * nh; i += kShThreads)  // every thread scales the entries that it wrote
    if (!(large >> (i % nh) & 1))
#pragma unroll
      for (int a = 0; a < NA; ++a) lut[(i % nh * NA + a) * n + i / nh] *= kLog2e;
  __syncthreads();
  return large;
}

// rows g and g + 8 of a 16-row tile of one head as an A operand, zeros past the segment
template <int D>
__device__ __forceinline__ void sh_rows(uint32_t (*a)[4], const uint16_t* src, const Params& p, int r, int qhi, int h,
                                        int lane) {
  load_a_rows<D>(a, r < qhi ? src + ((size_t)r * p.Hq + h) * D : nullptr,
                 r + 8 < qhi ? src + ((size_t)(r + 8) * p.Hq + h) * D : nullptr, lane);
}

// 16 rows of one head into a warp's buffer (zeros past the segment), and from there as an A operand
template <int D>
__device__ __forceinline__ int sh_piece(int row, int c) {
  return D == 32 ? row * 4 + (c ^ ((row >> 1) & 3)) : row * 8 + (c ^ (row & 7));
}
template <int D>
__device__ __forceinline__ void sh_copy(uint4* dst, const uint16_t* src, int row0, int n, int heads, int h, int lane) {
#pragma unroll
  for (int i = lane; i < 16 * (D / 8); i += 32) {
    const int r = i / (D / 8), c = i % (D / 8);
    const bool ok = r < n;
    cp_async16(dst + sh_piece<D>(r, c), src + ((size_t)(row0 + (ok ? r : 0)) * heads + h) * D + c * 8, ok);
  }
}
template <int D>
__device__ __forceinline__ void sh_take(uint32_t (*a)[4], const uint4* src, int lane) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
    ldmatrix_x4(a[ks][0], a[ks][1], a[ks][2], a[ks][3],
                smem_u32(src + sh_piece<D>(lane & 15, 2 * ks + (lane >> 4))));
}

// positions of rows r and r + 8 as the bias takes them, and the warp's range
template <int NA>
__device__ __forceinline__ void sh_row_positions(const Params& p, int r, int qhi, int (&rowc)[1][2][NA], int (&lo)[NA],
                                                 int (&hi)[NA]) {
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    const int x0 = p.pos_q[(size_t)min(r, qhi - 1) * NA + a], x1 = p.pos_q[(size_t)min(r + 8, qhi - 1) * NA + a];
    rowc[0][0][a] = p.maxd - x0;
    rowc[0][1][a] = p.maxd - x1;
    lo[a] = __reduce_min_sync(0xffffffffu, min(x0, x1));
    hi[a] = __reduce_max_sync(0xffffffffu, max(x0, x1));
    if (lo[a] < -kPosLimit || hi[a] > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
  }
}

template <int D, int NA>
__global__ void __launch_bounds__(kShThreads, 2) rp_short_fwd_kernel(const Params p) {
  using C = ShCfg<D, NA>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* ring = reinterpret_cast<uint4*>(smem_raw);  // [2][K, V]
  int* ps = reinterpret_cast<int*>(ring + 4 * C::kTile);
  float* lut = reinterpret_cast<float*>(smem_raw + C::kRing + C::kFlags);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  const ShPlace P = sh_place(p);
  if (!P.live) return;
  const int nk = P.khi - P.klo, blocks = (nk + kShKeys - 1) / kShKeys, top = 2 * p.maxd;
  const int tiles = (min(64, P.qhi - P.row0) + 15) / 16, units = P.nh * tiles;
  const int rounds = (units + kShWarps - 1) / kShWarps;
  // the blocks of all rounds, one after the other; a single block stays for good
  const int loads = blocks <= 1 ? blocks : rounds * blocks;
  auto load = [&](int i) {
    if (i < loads) {
      const int st = i & 1, k0 = P.klo + i % blocks * kShKeys, n = min(kShKeys, P.khi - k0);
      load_tile<D, kShKeys, kShThreads>(ring + st * 2 * C::kTile, p.k, k0, n, p.Hkv, P.hk, tid);
      load_tile<D, kShKeys, kShThreads>(ring + (st * 2 + 1) * C::kTile, p.v, k0, n, p.Hkv, P.hk, tid);
      for (int j = tid; j < kShKeys * NA; j += kShThreads)
        cp_async4(ps + st * kShKeys * NA + j, p.pos_k + (size_t)(k0 + min(j / NA, n - 1)) * NA + j % NA, true);
    }
    cp_async_commit();
  };
  load(0);
  uint32_t qa[1][D / 16][4];
  // units go row tile by row tile, so a warp that keeps its stride meets all heads of few tiles
  auto row_of = [&](int u) { return P.row0 + u / P.nh * 16 + g; };
  auto head_of = [&](int u) { return u % P.nh; };
  if (warp < units) sh_rows<D>(qa[0], p.q, p, row_of(warp), P.qhi, P.h0 + head_of(warp), lane);
  const uint32_t large = sh_fill<NA>(p, lut, P.h0, P.nh, tid);

  for (int round = 0; round < rounds; ++round) {
    const int u = round * kShWarps + warp;
    const bool work = u < units;
    const int r = row_of(work ? u : 0), hh = head_of(work ? u : 0);
    const float* mine = lut + hh * NA * (top + 1);
    const bool small = !(large >> hh & 1);
    const float mul = small ? p.scale * kLog2e : p.scale, to_log2 = small ? 1.0f : kLog2e;
    uint32_t nx[1][D / 16][4];
    if (u + kShWarps < units)
      sh_rows<D>(nx[0], p.q, p, row_of(u + kShWarps), P.qhi, P.h0 + head_of(u + kShWarps), lane);
    int rowc[1][2][NA], q_lo[NA], q_hi[NA];
    sh_row_positions<NA>(p, r, P.qhi, rowc, q_lo, q_hi);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;

    for (int blk = 0; blk < blocks; ++blk) {
      const int i = blocks == 1 ? 0 : round * blocks + blk;
      if (blocks > 1 || round == 0) {
        cp_async_wait<0>();
        __syncthreads();  // the block is here, and the other buffer's readers are done
        load(i + 1);
      }
      if (!work) continue;
      const uint4* kt = ring + (i & 1) * 2 * C::kTile;
      const uint4* vt = kt + C::kTile;
      const int* pt0 = ps + (i & 1) * kShKeys * NA;
#pragma unroll 1
      for (int kb = 0; kb < kShKeys; kb += kCols) {
        const int left = nk - blk * kShKeys - kb;
        if (left <= 0) break;
        const int* pt = pt0 + kb * NA;
        float s[1][kGroups][4];
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
          uint32_t b[D / 8];
          load_b_rows<D>(b, kt, kb, n, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][n][e] = 0.0f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(s[0][n], qa[0][d], b + 2 * d);
        }
        int mode[NA], one[NA];
#pragma unroll
        for (int a = 0; a < NA; ++a)
          mode[a] = axis_mode<NA>(pt + a, q_lo[a], q_hi[a], false, p.maxd, lane, one[a], p.status);
        float base[1][2];
        const bool fold = add_bias<NA, 1, 1>(s, base, mode, one, pt, mine, top, rowc, mul, !small, tq);
        if (left < kCols) {
          keep_branch();
#pragma unroll
          for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (tq * kLaneCols + 2 * n + e >= left) s[0][n][e] = s[0][n][2 + e] = -INFINITY;
        }
        float mx[2];
        bool need = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = fmaxf(s[0][0][2 * k], s[0][0][2 * k + 1]);
#pragma unroll
          for (int n = 1; n < kGroups; ++n) x = fmax3(x, s[0][n][2 * k], s[0][n][2 * k + 1]);
          mx[k] = fold ? fmaf(x, mul, base[0][k]) : x;
          need = need || mx[k] > m[k] + kShSlack;
        }
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float now = quad_max(fmaxf(mx[k], m[k]));
            const float f = m[k] == -INFINITY ? 0.0f : ex2((m[k] - now) * to_log2);
            m[k] = now;
            l[k] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][2 * k] *= f, o[n][2 * k + 1] *= f;
          }
        }
        uint32_t pa[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float ref = m[k] == -INFINITY ? 0.0f : m[k], cst = base[0][k] - ref;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            float p0 = s[0][n][2 * k], p1 = s[0][n][2 * k + 1];
            if (fold) {
              ffma2(p0, p1, p0, p1, mul, cst);
            } else {  // the subtraction first: exact for scores of any size
              fadd2_acc(p0, p1, -ref, -ref);
              if (!small) fmul2(p0, p1, p0, p1, kLog2e, kLog2e);
            }
            p0 = ex2(p0);
            p1 = ex2(p1);
            fadd2_acc(s0, s1, p0, p1);
            pa[n >> 1][(n & 1) * 2 + k] = pack2(p0, p1);
          }
          l[k] += s0 + s1;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int dc = 0; dc < D / 8; dc += 2) {
            uint32_t b[4];
            load_b_cols<D>(b, vt, kb, j, dc, lane);
            mma16816(o[dc], pa[j], b);
            mma16816(o[dc + 1], pa[j], b + 2);
          }
      }
    }
    if (work) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float sum = quad_sum(l[k]);
        const int row = r + 8 * k;
        if (row >= P.qhi) continue;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const size_t at = (size_t)row * p.Hq + P.h0 + hh;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<uint32_t*>(p.out + at * D + n * 8 + 2 * tq) =
              pack2(o[n][2 * k] * inv, o[n][2 * k + 1] * inv);
        if (tq == 0 && p.lse != nullptr)
          p.lse[at] = sum == 0.0f ? -INFINITY : (small ? m[k] * kLn2 : m[k]) + logf(sum);
      }
    }
    __syncwarp();
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) qa[0][d][e] = nx[0][d][e];
  }
}

template <int D, int NA>
__global__ void __launch_bounds__(kShThreads, D == 32 ? 2 : 1) rp_short_dq_kernel(const Params p) {
  using C = ShCfg<D, NA>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* ring = reinterpret_cast<uint4*>(smem_raw);  // [2][K, V]
  int* ps = reinterpret_cast<int*>(ring + 4 * C::kTile);
  uint4* next = reinterpret_cast<uint4*>(smem_raw + C::kRing) + (threadIdx.x >> 5) * 3 * C::kUnit;
  float* lut = reinterpret_cast<float*>(smem_raw + C::kRing + C::kUnits + C::kFlags);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  const ShPlace P = sh_place(p);
  if (!P.live) return;
  const int nk = P.khi - P.klo, blocks = (nk + kShKeys - 1) / kShKeys, top = 2 * p.maxd;
  const int tiles = (min(64, P.qhi - P.row0) + 15) / 16, units = P.nh * tiles;
  const int rounds = (units + kShWarps - 1) / kShWarps;
  const int loads = blocks <= 1 ? blocks : rounds * blocks;
  auto load = [&](int i) {
    if (i < loads) {
      const int st = i & 1, k0 = P.klo + i % blocks * kShKeys, n = min(kShKeys, P.khi - k0);
      load_tile<D, kShKeys, kShThreads>(ring + st * 2 * C::kTile, p.k, k0, n, p.Hkv, P.hk, tid);
      load_tile<D, kShKeys, kShThreads>(ring + (st * 2 + 1) * C::kTile, p.v, k0, n, p.Hkv, P.hk, tid);
      for (int j = tid; j < kShKeys * NA; j += kShThreads)
        cp_async4(ps + st * kShKeys * NA + j, p.pos_k + (size_t)(k0 + min(j / NA, n - 1)) * NA + j % NA, true);
    }
    cp_async_commit();
  };
  load(0);
  auto row_of = [&](int u) { return P.row0 + u / P.nh * 16 + g; };
  auto head_of = [&](int u) { return u % P.nh; };
  // a unit's operands: queries, dO and out by asynchronous copies, LSE
  float next_lse[2];
  auto fetch = [&](int u) {
    if (u < units) {
      const int r0 = P.row0 + u / P.nh * 16, r = r0 + g, n = P.qhi - r0, h = P.h0 + head_of(u);
      sh_copy<D>(next, p.q, r0, n, p.Hq, h, lane);
      sh_copy<D>(next + C::kUnit, p.dout, r0, n, p.Hq, h, lane);
      sh_copy<D>(next + 2 * C::kUnit, p.o_in, r0, n, p.Hq, h, lane);
      next_lse[0] = r < P.qhi ? p.lse_in[(size_t)r * p.Hq + h] : INFINITY;
      next_lse[1] = r + 8 < P.qhi ? p.lse_in[(size_t)(r + 8) * p.Hq + h] : INFINITY;
    }
    cp_async_commit();
  };
  fetch(warp);
  const uint32_t large = sh_fill<NA>(p, lut, P.h0, P.nh, tid);

  for (int round = 0; round < rounds; ++round) {
    const int u = round * kShWarps + warp;
    const bool work = u < units;
    const int r = row_of(work ? u : 0), hh = head_of(work ? u : 0), h = P.h0 + hh;
    const float* mine = lut + hh * NA * (top + 1);
    const bool small = !(large >> hh & 1);
    const float mul = small ? p.scale * kLog2e : p.scale;
    uint32_t qa[D / 16][4], da[D / 16][4], oa[D / 16][4];
    cp_async_wait<0>();
    __syncwarp();
    if (work) {
      sh_take<D>(qa, next, lane);
      sh_take<D>(da, next + C::kUnit, lane);
      sh_take<D>(oa, next + 2 * C::kUnit, lane);
    }
    const float lse[2] = {work ? row_lse(next_lse[0]) : INFINITY, work ? row_lse(next_lse[1]) : INFINITY};
    __syncwarp();
    fetch(u + kShWarps);
    int rowc[1][2][NA], q_lo[NA], q_hi[NA];
    sh_row_positions<NA>(p, r, P.qhi, rowc, q_lo, q_hi);
    float delta[2] = {0.0f, 0.0f}, rest[2] = {0.0f, 0.0f}, l[2] = {0.0f, 0.0f}, row[2];
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = bf16_to_f32((uint16_t)da[d][e]) * bf16_to_f32((uint16_t)oa[d][e]);
        delta[e & 1] += fmaf(__uint_as_float(da[d][e] & 0xffff0000u), __uint_as_float(oa[d][e] & 0xffff0000u), lo);
      }
    bool huge = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      delta[k] = quad_sum(delta[k]);
      huge = huge || is_huge(lse[k]);
      row[k] = row_const(lse[k], small);
    }
    const bool exact = !small || __any_sync(0xffffffffu, huge);
    float dq[D / 8][4], pk[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dq[n][e] = pk[n][e] = 0.0f;

    for (int blk = 0; blk < blocks; ++blk) {
      const int i = blocks == 1 ? 0 : round * blocks + blk;
      if (blocks > 1 || round == 0) {
        if (blocks == 1)
          cp_async_wait<1>();  // all but the next operands
        else
          cp_async_wait<0>();
        __syncthreads();  // the block is here, and the other buffer's readers are done
        load(i + 1);
      }
      if (!work) continue;
      const uint4* kt = ring + (i & 1) * 2 * C::kTile;
      const uint4* vt = kt + C::kTile;
      const int* pt0 = ps + (i & 1) * kShKeys * NA;
#pragma unroll 1
      for (int kb = 0; kb < kShKeys; kb += kCols) {
        const int left = nk - blk * kShKeys - kb;
        if (left <= 0) break;
        const int* pt = pt0 + kb * NA;
        float s[1][kGroups][4], dp[kGroups][4];
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
          uint32_t b[D / 8];
          load_b_rows<D>(b, kt, kb, n, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][n][e] = dp[n][e] = 0.0f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(s[0][n], qa[d], b + 2 * d);
          load_b_rows<D>(b, vt, kb, n, lane);
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(dp[n], da[d], b + 2 * d);
        }
        int mode[NA], one[NA];
#pragma unroll
        for (int a = 0; a < NA; ++a)
          mode[a] = axis_mode<NA>(pt + a, q_lo[a], q_hi[a], false, p.maxd, lane, one[a], p.status);
        float base[1][2];
        const bool fold = add_bias<NA, 1, 1>(s, base, mode, one, pt, mine, top, rowc, mul, exact, tq);
        if (left < kCols) {
          keep_branch();
#pragma unroll
          for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (tq * kLaneCols + 2 * n + e >= left) s[0][n][e] = s[0][n][2 + e] = -INFINITY;
        }
        uint32_t sa[2][4], pa[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float cst = base[0][k] - row[k];
          float s0 = 0.0f, s1 = 0.0f, l0 = 0.0f, l1 = 0.0f;
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            float p0 = s[0][n][2 * k], p1 = s[0][n][2 * k + 1];
            if (fold) {
              ffma2(p0, p1, p0, p1, mul, cst);
            } else {  // the subtraction first: exact for scores of any size
              fadd2_acc(p0, p1, -row[k], -row[k]);
              if (!small) fmul2(p0, p1, p0, p1, kLog2e, kLog2e);
            }
            p0 = ex2(p0);
            p1 = ex2(p1);
            fadd2_acc(l0, l1, p0, p1);
            pa[n >> 1][(n & 1) * 2 + k] = pack2(p0, p1);
            float d0 = dp[n][2 * k], d1 = dp[n][2 * k + 1];
            fadd2_acc(d0, d1, -delta[k], -delta[k]);
            fmul2(d0, d1, d0, d1, p0, p1);
            fadd2_acc(s0, s1, d0, d1);
            sa[n >> 1][(n & 1) * 2 + k] = pack2(d0, d1);
          }
          rest[k] += s0 + s1;
          l[k] += l0 + l1;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int dc = 0; dc < D / 8; dc += 2) {
            uint32_t b[4];
            load_b_cols<D>(b, kt, kb, j, dc, lane);
            mma16816(dq[dc], sa[j], b);
            mma16816(dq[dc + 1], sa[j], b + 2);
            mma16816(pk[dc], pa[j], b);
            mma16816(pk[dc + 1], pa[j], b + 2);
          }
      }
    }
    if (work) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float sum = quad_sum(l[k]), parts = quad_sum(rest[k]);
        const int at_row = r + 8 * k;
        if (at_row >= P.qhi) continue;
        const float inv = row_inverse(sum, row[k], p.status), corr = row_corr(sum);
        const float more = parts * inv;  // Delta less the one of the saved out
        const size_t at = (size_t)at_row * p.Hq + h;
        if (tq == 0) {
          p.delta[at] = delta[k] + more;
          p.lse2[at] = row_lse2(row[k], small, corr);
          p.corr[at] = corr;
        }
        const float f = inv * p.scale;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<uint32_t*>(p.dq + at * D + n * 8 + 2 * tq) =
              pack2(fmaf(-more, pk[n][2 * k], dq[n][2 * k]) * f, fmaf(-more, pk[n][2 * k + 1], dq[n][2 * k + 1]) * f);
      }
    }
  }
}

template <int D, int NA>
static lsrm_status run_short(const Params& p, long long ctas, bool dq, cudaStream_t s) {
  const size_t bytes = ShCfg<D, NA>::smem(p.maxd, p.G < kShHeads ? p.G : kShHeads, dq);
  const void* kernel = dq ? (const void*)rp_short_dq_kernel<D, NA> : (const void*)rp_short_fwd_kernel<D, NA>;
  if (!allow_smem(kernel, bytes)) return LSRM_ERR_CUDA;
  if (dq)
    rp_short_dq_kernel<D, NA><<<(unsigned)ctas, kShThreads, bytes, s>>>(p);
  else
    rp_short_fwd_kernel<D, NA><<<(unsigned)ctas, kShThreads, bytes, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

lsrm_status launch_short(const Params& p, int D, int NA, long long ctas, bool dq, cudaStream_t s) {
  if (D == 32)
    return NA == 1 ? run_short<32, 1>(p, ctas, dq, s) : NA == 2 ? run_short<32, 2>(p, ctas, dq, s)
                                                                : run_short<32, 3>(p, ctas, dq, s);
  return NA == 1 ? run_short<64, 1>(p, ctas, dq, s) : NA == 2 ? run_short<64, 2>(p, ctas, dq, s)
                                                              : run_short<64, 3>(p, ctas, dq, s);
}

}  // namespace rp
}  // namespace lsrm
