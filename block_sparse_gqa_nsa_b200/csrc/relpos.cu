// Forward of the attention with a learned relative position bias by buckets (relpos.cuh has the
// formulas).
//
// Each score costs one exponential, a table look-up per axis and 4 d tensor FLOP, so at d = 32 / 64 the
// per-score work of the softmax warps, not the tensor pipe, is the bound.  fwd_plan chooses among four
// kernels by how many query rows share a key stream:
//   * rp_few_kernel (here): 16 rows (tokens x heads of one KV group) a CTA, each warp its own keys, the
//     warps joined in shared memory: single tokens and other short query runs, bound by reading K, V.  64 single
//     tokens against ragged pasts of up to 8192 (32 heads of 32) 25 us, 72 MB of K and V at 2.9 TB/s;
//   * rp_short_fwd_kernel (relpos_short.cu): many short segments;
//   * rp_fwd_kernel (here): 64 or 128 queries of one head a CTA, 32 a warp, some tens of queries a segment: keys
//     stream through shared memory in chunks of 64 (cp.async, three stages), scores stay in registers from
//     Q K^T to P V (mma.sync row tiles: a lane sees its rows' distances directly, and P goes from the
//     accumulator layout to the operand layout without leaving the registers; tcgen05's 128-row tiles would be
//     half empty);
//   * rp_fwd_tc_kernel (relpos_tc.cu): 256 queries a CTA on tcgen05.
// All but the second split the keys over CTAs when there are too few rows to fill the GPU; rp_join_kernel then
// adds the parts by their softmax references and sums in a fixed order.
//
// The softmax keeps a reference per row that moves only when a score exceeds it by more than 8 in the table's
// units (P stays below e^8, far inside fp32 and bf16), so most tiles need no rescaling and no shuffles.
// Row sums are fp32 over the unrounded P; P is rounded to bf16 for the second product, as its
// operand V is bf16.
#include "relpos.cuh"

namespace lsrm {
namespace rp {

constexpr int kChunk = 64;  // keys a stage
constexpr int kStages = 3;
constexpr float kSlack = 8.0f;

template <int D, int NA, int NW>
struct FwdCfg {
  // CTAs of 128 threads an SM.  16 and 64 segments of 24 to 64 queries against 512 keys, 32 heads of 32: 41-43 us
  // and 112-121; four CTAs (fewer registers) 50-57; score tiles of 64 columns and two CTAs 33-60 and 118-123.
  static constexpr int kMinCtas = (D == 32 ? 3 : 2) * 4 / NW;
  static constexpr int kRows = 32 * NW, kThreads = 32 * NW;
  static constexpr int kTile = kChunk * D / 8;  // 16-byte pieces of a K or V stage
  static constexpr size_t kFixed = (size_t)kStages * (2 * kTile * 16 + kChunk * NA * 4);
  static size_t smem(int maxd) { return kFixed + (size_t)NA * (2 * maxd + 1) * 4; }
};

// The softmax references and sums of a warp's rows (MT row tiles of 16), in the table's units (to_log2: their
// factor to log2); mx is the lane's largest score per row.  Where one passes the reference by more than kSlack,
// the tile's references move to their rows' maxima and the sums and outputs are rescaled.
template <int MT>
struct RowState {
  float m[MT][2], l[MT][2];
};
template <int MT, int ND>
__device__ __forceinline__ void move_reference(RowState<MT>& st, float (&o)[MT][ND][4], const float (&mx)[MT][2],
                                               float to_log2) {
  bool need = false;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) need |= mx[mt][i] > st.m[mt][i] + kSlack;
  if (!__any_sync(0xffffffffu, need)) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float m = quad_max(fmaxf(mx[mt][i], st.m[mt][i]));
      const float f = st.m[mt][i] == -INFINITY ? 0.0f : ex2((st.m[mt][i] - m) * to_log2);
      st.m[mt][i] = m;
      st.l[mt][i] *= f;
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        o[mt][n][2 * i] *= f;
        o[mt][n][2 * i + 1] *= f;
      }
    }
}

template <int D, int NA, int NW>
__global__ void __launch_bounds__(32 * NW, FwdCfg<D, NA, NW>::kMinCtas) rp_fwd_kernel(const Params p) {
  using C = FwdCfg<D, NA, NW>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4* ks = reinterpret_cast<uint4*>(smem_raw);
  uint4* vs = ks + kStages * C::kTile;
  int* ps = reinterpret_cast<int*>(vs + kStages * C::kTile);
  float* lut = reinterpret_cast<float*>(ps + kStages * kChunk * NA);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  let_dependents();
  int unit = blockIdx.x;
  const int split = unit % p.splits;
  unit /= p.splits;
  const int h = unit % p.Hq, tile = unit / p.Hq, hk = h / p.G;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, C::kRows, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + (tile - first) * C::kRows;
  if (tile < first || row0 >= qhi) return;
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int nk = khi - klo, chunks = (nk + kChunk - 1) / kChunk;
  const int per = (chunks + p.splits - 1) / p.splits;
  const int c0 = min(split * per, chunks), c1 = min(c0 + per, chunks);
  const int top = 2 * p.maxd;

  auto load = [&](int c) {
    if (c < c1) {
      const int st = c % kStages, k0 = klo + c * kChunk, n = min(kChunk, khi - k0);
      load_tile<D, kChunk, C::kThreads>(ks + st * C::kTile, p.k, k0, n, p.Hkv, hk, tid);
      load_tile<D, kChunk, C::kThreads>(vs + st * C::kTile, p.v, k0, n, p.Hkv, hk, tid);
      // positions past the end repeat the last key's, so they do not widen the tile's range
      for (int i = tid; i < kChunk * NA; i += C::kThreads)
        cp_async4(ps + st * kChunk * NA + i, p.pos_k + (size_t)(k0 + min(i / NA, n - 1)) * NA + i % NA, true);
    }
    cp_async_commit();
  };
  load(c0);
  load(c0 + 1);
  // (a row's reference and sums are in the table's units)
  const bool small = fill_units<NA, C::kThreads>(p, lut, h, tid);
  const float mul = small ? p.scale * kLog2e : p.scale, to_log2 = small ? 1.0f : kLog2e;

  // the warp's 32 rows: operands, positions and their range
  uint32_t qa[2][D / 16][4];
  int qp[2][2][NA], q_lo[NA], q_hi[NA];
  const int wrow = row0 + warp * 32;
#pragma unroll
  for (int a = 0; a < NA; ++a) q_lo[a] = INT32_MAX, q_hi[a] = INT32_MIN;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    const int r = wrow + mt * 16 + g;
    load_a_rows<D>(qa[mt], r < qhi ? p.q + ((size_t)r * p.Hq + h) * D : nullptr,
                   r + 8 < qhi ? p.q + ((size_t)(r + 8) * p.Hq + h) * D : nullptr, lane);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int x = p.pos_q[(size_t)min(r + 8 * i, qhi - 1) * NA + a];
        qp[mt][i][a] = p.maxd - x;
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

  RowState<2> st;
  float o[2][D / 8][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) st.m[mt][i] = -INFINITY, st.l[mt][i] = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.0f;
  }

  for (int c = c0; c < c1; ++c) {
    cp_async_wait<1>();
    __syncthreads();
    load(c + 2);  // into the stage read before the barrier
    const uint4* kt = ks + (c % kStages) * C::kTile;
    const uint4* vt = vs + (c % kStages) * C::kTile;
    const int* pt = ps + (c % kStages) * kChunk * NA;
#pragma unroll 1
    for (int kb = 0; kb < kChunk; kb += kCols) {
      const int left = nk - c * kChunk - kb;  // keys from here on
      if (left <= 0 || wrow >= qhi) break;
      float s[2][kGroups][4];
#pragma unroll
      for (int n = 0; n < kGroups; ++n) {
        uint32_t b[D / 8];
        load_b_rows<D>(b, kt, kb, n, lane);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][n][e] = 0.0f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) mma16816(s[mt][n], qa[mt][d], b + 2 * d);
        }
      }
      int mode[NA], one[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a)
        mode[a] = axis_mode<NA>(pt + kb * NA + a, q_lo[a], q_hi[a], false, p.maxd, lane, one[a], p.status);
      float base[2][2];
      const bool fold = add_bias<NA, 2, 1>(s, base, mode, one, pt + kb * NA, lut, top, qp, mul, !small, tq);
      if (left < kCols) {
        keep_branch();
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (tq * kLaneCols + 2 * n + e >= left)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) s[mt][n][e] = s[mt][n][2 + e] = -INFINITY;
      }
      float mx[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmax3(s[mt][0][2 * i], s[mt][0][2 * i + 1], s[mt][1][2 * i]);
          x = fmaxf(x, s[mt][1][2 * i + 1]);
#pragma unroll
          for (int n = 2; n < kGroups; ++n) x = fmax3(x, s[mt][n][2 * i], s[mt][n][2 * i + 1]);
          mx[mt][i] = fold ? fmaf(x, mul, base[mt][i]) : x;
        }
      move_reference<2, D / 8>(st, o, mx, to_log2);
      // P = exp(t - m): with the bias in the scores the subtraction comes first (exact for equal scores
      // of any size); with a bias common to a row everything folds into one multiply-add
      uint32_t pa[2][kGroups / 2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m = st.m[mt][i] == -INFINITY ? 0.0f : st.m[mt][i];
          const float cst = base[mt][i] - m;
          float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
          for (int n = 0; n < kGroups; ++n) {
            float p0 = s[mt][n][2 * i], p1 = s[mt][n][2 * i + 1];
            if (fold) {
              ffma2(p0, p1, p0, p1, mul, cst);
            } else {
              fadd2_acc(p0, p1, -m, -m);
              if (!small) fmul2(p0, p1, p0, p1, kLog2e, kLog2e);
            }
            p0 = ex2(p0);
            p1 = ex2(p1);
            fadd2_acc(sum0, sum1, p0, p1);
            pa[mt][n >> 1][(n & 1) * 2 + i] = pack2(p0, p1);
          }
          st.l[mt][i] += sum0 + sum1;
        }
#pragma unroll
      for (int j = 0; j < kGroups / 2; ++j)
#pragma unroll
        for (int dc = 0; dc < D / 8; dc += 2) {
          uint32_t b[4];
          load_b_cols<D>(b, vt, kb, j, dc, lane);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            mma16816(o[mt][dc], pa[mt][j], b);
            mma16816(o[mt][dc + 1], pa[mt][j], b + 2);
          }
        }
    }
  }

#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float l = quad_sum(st.l[mt][i]);
      const int r = wrow + mt * 16 + g + 8 * i;
      if (r >= qhi) continue;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float ref = small ? st.m[mt][i] * kLn2 : st.m[mt][i];
      const float lse = l == 0.0f ? -INFINITY : ref + logf(l);
      const size_t at = (size_t)r * p.Hq + h;
      if (p.splits == 1) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<uint32_t*>(p.out + at * D + n * 8 + 2 * tq) =
              pack2(o[mt][n][2 * i] * inv, o[mt][n][2 * i + 1] * inv);
        if (tq == 0 && p.lse != nullptr) p.lse[at] = lse;
      } else {
        const size_t pat = (size_t)split * p.Nq * p.Hq + at;
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(p.o_part + pat * D + n * 8 + 2 * tq) =
              make_float2(o[mt][n][2 * i] * inv, o[mt][n][2 * i + 1] * inv);
        if (tq == 0) p.ml_part[pat] = make_float2(ref, l);
      }
    }
}

// ---- few rows a key stream -----------------------------------------------------------------------

constexpr int kFewWarps = 4, kFewThreads = 32 * kFewWarps, kFewKeys = 32;

template <int D, int NA>
struct FewCfg {
  static constexpr int kTile = kFewKeys * D / 8;
  static constexpr size_t kRing = (size_t)kFewWarps * kStages * (2 * kTile * 16 + kFewKeys * NA * 4);
  static constexpr size_t kJoin = (size_t)kFewWarps * 16 * (D + 2) * 4;  // laid over the ring
  static_assert(kJoin <= kRing, "the warps' join lies over the key ring");
  static size_t smem(int maxd, int nb, int gh) {
    return kRing + (size_t)NA * nb * gh * 4 + (((size_t)2 * maxd + 1 + 15) & ~(size_t)15);
  }
};

template <int D, int NA>
__global__ void __launch_bounds__(kFewThreads) rp_few_kernel(const Params p) {
  using C = FewCfg<D, NA>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
  const int GH = min(p.G, 16), T = 16 / GH, hgroups = (p.G + GH - 1) / GH;
  uint4* ring = reinterpret_cast<uint4*>(smem_raw) + (size_t)warp * kStages * 2 * C::kTile;
  int* ps = reinterpret_cast<int*>(smem_raw + (size_t)kFewWarps * kStages * 2 * C::kTile * 16) +
            warp * kStages * kFewKeys * NA;
  float* tab = reinterpret_cast<float*>(smem_raw + C::kRing);  // [NA][NB][GH]
  uint8_t* bk = reinterpret_cast<uint8_t*>(tab + NA * p.NB * GH);

  let_dependents();
  int unit = blockIdx.x;
  const int split = unit % p.splits;
  unit /= p.splits;
  const int hg = unit % hgroups;
  unit /= hgroups;
  const int hk = unit % p.Hkv, tile = unit / p.Hkv;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, T, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + (tile - first) * T;
  if (tile < first || row0 >= qhi) return;
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int nk = khi - klo, chunks = (nk + kFewKeys - 1) / kFewKeys;
  const int per = (chunks + p.splits - 1) / p.splits;
  const int c0 = min(split * per, chunks), c1 = min(c0 + per, chunks);
  const int top = 2 * p.maxd, h0 = hk * p.G + hg * GH, nh = min(GH, p.G - hg * GH);

  auto load = [&](int c) {
    if (c < c1) {
      const int st = ((c - c0) / kFewWarps) % kStages, k0 = klo + c * kFewKeys, n = min(kFewKeys, khi - k0);
      load_tile<D, kFewKeys, 32>(ring + st * 2 * C::kTile, p.k, k0, n, p.Hkv, hk, lane);
      load_tile<D, kFewKeys, 32>(ring + (st * 2 + 1) * C::kTile, p.v, k0, n, p.Hkv, hk, lane);
#pragma unroll
      for (int i = lane; i < kFewKeys * NA; i += 32)
        cp_async4(ps + st * kFewKeys * NA + i, p.pos_k + (size_t)(k0 + min(i / NA, n - 1)) * NA + i % NA, true);
    }
    cp_async_commit();
  };
  load(c0 + warp);
  load(c0 + warp + kFewWarps);

  for (int i = tid; i < top + 1; i += kFewThreads) {
    const int b = checked_bucket(p, i);
    bk[i] = (uint8_t)(b < 0 ? 255 : b);
  }
  // the heads' tables, in log2 units when every entry is small or -inf (fill_units)
  bool mine_small = true;
  for (int i = tid; i < NA * p.NB * GH; i += kFewThreads) {
    const int hh = i % GH;
    const float x = hh < nh ? bf16_to_f32(p.table[(size_t)(i / GH) * p.Hq + h0 + hh]) : 0.0f;
    mine_small = mine_small && (fabsf(x) <= kSmallBias || x == -INFINITY);
    tab[i] = x;
  }
  const bool small = __syncthreads_and(mine_small);
  if (small)  // every thread scales the entries that it wrote
    for (int i = tid; i < NA * p.NB * GH; i += kFewThreads) tab[i] *= kLog2e;
  const float mul = small ? p.scale * kLog2e : p.scale, to_log2 = small ? 1.0f : kLog2e;

  // rows g and g + 8: (token, head) pairs
  uint32_t qa[D / 16][4];
  int qp[2][NA], q_lo[NA], q_hi[NA], hh[2];
  size_t at[2];
  bool live[2];
#pragma unroll
  for (int a = 0; a < NA; ++a) q_lo[a] = INT32_MAX, q_hi[a] = INT32_MIN;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i, t = r / GH;
    hh[i] = r % GH;
    live[i] = t < T && row0 + t < qhi && hh[i] < nh;
    at[i] = (size_t)(row0 + t) * p.Hq + h0 + hh[i];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int x = p.pos_q[(size_t)min(row0 + t, qhi - 1) * NA + a];
      qp[i][a] = p.maxd - x;
      q_lo[a] = min(q_lo[a], x);
      q_hi[a] = max(q_hi[a], x);
    }
  }
  load_a_rows<D>(qa, live[0] ? p.q + at[0] * D : nullptr, live[1] ? p.q + at[1] * D : nullptr, lane);
#pragma unroll
  for (int a = 0; a < NA; ++a) {
    q_lo[a] = __reduce_min_sync(0xffffffffu, q_lo[a]);
    q_hi[a] = __reduce_max_sync(0xffffffffu, q_hi[a]);
    if (q_lo[a] < -kPosLimit || q_hi[a] > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
  }
  __syncthreads();

  auto bias_at = [&](int a, int idx, int head) {
    const int b = bk[idx];
    return b == 255 ? 0.0f : tab[(a * p.NB + b) * GH + head];
  };
  RowState<1> st;
  float o[1][D / 8][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) st.m[0][i] = -INFINITY, st.l[0][i] = 0.0f;
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[0][n][e] = 0.0f;

  for (int c = c0 + warp; c < c1; c += kFewWarps) {
    cp_async_wait<1>();
    __syncwarp();
    load(c + 2 * kFewWarps);
    const int sg = ((c - c0) / kFewWarps) % kStages;
    const uint4* kt = ring + sg * 2 * C::kTile;
    const uint4* vt = kt + C::kTile;
    const int* pt = ps + sg * kFewKeys * NA;
    const int left = nk - c * kFewKeys;
    float s[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      uint32_t b[D / 8];
      load_b_rows<D>(b, kt, 0, n, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) mma16816(s[n], qa[d], b + 2 * d);
    }
    float ub[2] = {0.0f, 0.0f};
    int uni[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int x = pt[lane * NA + a];
      const int lo = __reduce_min_sync(0xffffffffu, x), hi = __reduce_max_sync(0xffffffffu, x);
      if (lo < -kPosLimit || hi > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
      const int near = clamp_index(lo - q_hi[a], p.maxd, top), far = clamp_index(hi - q_lo[a], p.maxd, top);
      uni[a] = near == far ? near : -1;
      if (uni[a] >= 0 && small) {
        ub[0] += bias_at(a, uni[a], hh[0]);
        ub[1] += bias_at(a, uni[a], hh[1]);
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) ffma2(s[n][2 * i], s[n][2 * i + 1], s[n][2 * i], s[n][2 * i + 1], mul, ub[i]);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      if (uni[a] >= 0 && small) continue;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int x = pt[(tq * 8 + 2 * n + e) * NA + a];
#pragma unroll
          for (int i = 0; i < 2; ++i) s[n][2 * i + e] += bias_at(a, clamp_index(x, qp[i][a], top), hh[i]);
        }
    }
    if (left < kFewKeys) {
      keep_branch();
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (tq * 8 + 2 * n + e >= left) s[n][e] = s[n][2 + e] = -INFINITY;
    }
    float mx[1][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
      for (int n = 1; n < 4; ++n) x = fmax3(x, s[n][2 * i], s[n][2 * i + 1]);
      mx[0][i] = x;
    }
    move_reference<1, D / 8>(st, o, mx, to_log2);
    uint32_t pa[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float m = st.m[0][i] == -INFINITY ? 0.0f : st.m[0][i];
      float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {  // the subtraction first: exact for scores of any size
        float a = s[n][2 * i], b = s[n][2 * i + 1];
        fadd2_acc(a, b, -m, -m);
        if (!small) fmul2(a, b, a, b, kLog2e, kLog2e);
        a = ex2(a);
        b = ex2(b);
        fadd2_acc(sum0, sum1, a, b);
        pa[n >> 1][(n & 1) * 2 + i] = pack2(a, b);
      }
      st.l[0][i] += sum0 + sum1;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int dc = 0; dc < D / 8; dc += 2) {
        uint32_t b[4];
        load_b_cols<D>(b, vt, 0, j, dc, lane);
        mma16816(o[0][dc], pa[j], b);
        mma16816(o[0][dc + 1], pa[j], b + 2);
      }
    __syncwarp();
  }

  // join the warps: [warp][row][D] outputs, then references and sums, over the key ring
  cp_async_wait<0>();
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem_raw);
  float* jm = jo + kFewWarps * 16 * D;
  float* jl = jm + kFewWarps * 16;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float l = quad_sum(st.l[0][i]);
    const int r = warp * 16 + g + 8 * i;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(jo + r * D + n * 8 + 2 * tq) = make_float2(o[0][n][2 * i], o[0][n][2 * i + 1]);
    if (tq == 0) {
      jm[r] = st.m[0][i];
      jl[r] = l;
    }
  }
  __syncthreads();
  for (int i = tid; i < 16 * (D / 2); i += kFewThreads) {
    const int r = i / (D / 2), d = i % (D / 2) * 2, t = r / GH, head = r % GH;
    if (t >= T || row0 + t >= qhi || head >= nh) continue;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, jm[w * 16 + r]);
    float l = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float mw = jm[w * 16 + r];
      const float f = mw == -INFINITY && jl[w * 16 + r] == 0.0f ? 0.0f : ex2((mw - m) * to_log2);
      l = fmaf(f, jl[w * 16 + r], l);
      x = fmaf(f, jo[(w * 16 + r) * D + d], x);
      y = fmaf(f, jo[(w * 16 + r) * D + d + 1], y);
    }
    const float ref = small ? m * kLn2 : m;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l, lse = l == 0.0f ? -INFINITY : ref + logf(l);
    const size_t to = (size_t)(row0 + t) * p.Hq + h0 + head;
    if (p.splits == 1) {
      *reinterpret_cast<uint32_t*>(p.out + to * D + d) = pack2(x * inv, y * inv);
      if (d == 0 && p.lse != nullptr) p.lse[to] = lse;
    } else {
      const size_t pat = (size_t)split * p.Nq * p.Hq + to;
      *reinterpret_cast<float2*>(p.o_part + pat * D + d) = make_float2(x * inv, y * inv);
      if (d == 0) p.ml_part[pat] = make_float2(ref, l);
    }
  }
}

// ---- parts of a split -----------------------------------------------------------------------------

constexpr int kJoinRows = 1, kJoinThreads = 256;

// out = sum_s l_s exp(m_s - m) o_s / sum_s l_s exp(m_s - m) in the order of the splits (reference and
// sum apart: their LSE would lose the sum beside a huge reference); D / 4 lanes a (query, head)
template <int D>
__global__ void __launch_bounds__(kJoinThreads) rp_join_kernel(const Params p) {
  int first, qlo, qhi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, kJoinRows, blockIdx.x, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + ((int)blockIdx.x - first) * kJoinRows;
  wait_for_previous();
  if ((int)blockIdx.x < first || row0 >= qhi) return;
  const int rows = min(kJoinRows, qhi - row0);
  const size_t stride = (size_t)p.Nq * p.Hq;
  for (int i = threadIdx.x; i < rows * p.Hq * (D / 4); i += kJoinThreads) {
    const size_t at = (size_t)row0 * p.Hq + i / (D / 4);
    const int d = i % (D / 4) * 4;
    float m = -INFINITY;
    for (int s = 0; s < p.splits; ++s) m = fmaxf(m, p.ml_part[s * stride + at].x);
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < p.splits; ++s) {
      const float2 ml = p.ml_part[s * stride + at];
      if (ml.y == 0.0f) continue;  // no key
      const float f = ml.y * ex2((ml.x - m) * kLog2e);
      const float4 x = *reinterpret_cast<const float4*>(p.o_part + (s * stride + at) * D + d);
      l += f;
      o.x = fmaf(f, x.x, o.x);
      o.y = fmaf(f, x.y, o.y);
      o.z = fmaf(f, x.z, o.z);
      o.w = fmaf(f, x.w, o.w);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(p.out + at * D + d) =
        make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    if (d == 0 && p.lse != nullptr) p.lse[at] = l == 0.0f ? -INFINITY : m + logf(l);
  }
}

// ---- launch ---------------------------------------------------------------------------------------

static lsrm_status launched() { return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA; }

template <int D, int NA, int NW>
static lsrm_status run_fwd(const Params& p, long long ctas, cudaStream_t s) {
  const size_t bytes = FwdCfg<D, NA, NW>::smem(p.maxd);
  if (!allow_smem(rp_fwd_kernel<D, NA, NW>, bytes)) return LSRM_ERR_CUDA;
  rp_fwd_kernel<D, NA, NW><<<(unsigned)ctas, 32 * NW, bytes, s>>>(p);
  return launched();
}

lsrm_status launch_fwd_tc(const Params& p, int D, int NA, long long ctas, cudaStream_t s);
lsrm_status launch_short(const Params& p, int D, int NA, long long ctas, bool dq, cudaStream_t s);

template <int D, int NA>
static lsrm_status run_shape(const Params& p, const FwdPlan& f, cudaStream_t s) {
  lsrm_status st;
  if (f.rows < 0) {
    st = launch_short(p, D, NA, f.ctas, false, s);
  } else if (f.rows == 0) {
    const size_t bytes = FewCfg<D, NA>::smem(p.maxd, p.NB, p.G < 16 ? p.G : 16);
    if (!allow_smem(rp_few_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
    rp_few_kernel<D, NA><<<(unsigned)f.ctas, kFewThreads, bytes, s>>>(p);
    st = launched();
  } else if (f.rows == 256) {
    st = launch_fwd_tc(p, D, NA, f.ctas, s);
  } else if (f.rows == 64) {
    st = run_fwd<D, NA, 2>(p, f.ctas, s);
  } else if constexpr (D == 32) {  // (fwd_plan: 128 rows at head dim 32 only)
    st = run_fwd<D, NA, 4>(p, f.ctas, s);
  } else {
    return LSRM_ERR_UNSUPPORTED;
  }
  if (st != LSRM_OK || f.splits == 1) return st;
  return launch_dependent(rp_join_kernel<D>, dim3((unsigned)(p.Nq / kJoinRows + p.S)), kJoinThreads, s, p)
             ? LSRM_OK
             : LSRM_ERR_CUDA;
}

}  // namespace rp

lsrm_status launch_relpos_forward(const rp::Params& p, int D, int NA, const rp::FwdPlan& f, cudaStream_t s) {
  using namespace rp;
  if (D == 32) {
    if (NA == 1) return run_shape<32, 1>(p, f, s);
    if (NA == 2) return run_shape<32, 2>(p, f, s);
    return run_shape<32, 3>(p, f, s);
  }
  if (NA == 1) return run_shape<64, 1>(p, f, s);
  if (NA == 2) return run_shape<64, 2>(p, f, s);
  return run_shape<64, 3>(p, f, s);
}

}  // namespace lsrm
