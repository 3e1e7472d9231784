// Forward of the attention with a learned relative position bias by buckets on the 5th-generation
// tensor cores (relpos.cuh has the formulas): the kernel of long query runs.
//
// One CTA = 256 queries of one head, as two row tiles of 128 (one query a tensor-memory lane), against
// the keys of their segment in chunks of 64.  Roles (320 threads, two CTAs an SM): warp 0 brings K and V
// by TMA and the keys' positions by plain loads, and notes what each chunk's positions have in common;
// warp 1 issues the MMAs (S = Q K^T from shared memory into tensor memory, O += P V with P read from
// tensor memory); warps 2-5 and 6-9 are the softmax threads of the two tiles, one query each.
//
// A thread owns a row, so a bias that is the same for a run of keys costs one look-up for the run: per
// axis a chunk lies on one clamped distance (no look-up), on one position per 16 keys, per 4 keys, or has
// a look-up per score.  At d = 32 a score's exponential (16 a clock and SM) costs as much as 256 tensor
// FLOP, so the softmax threads are the bound: packed fp32 pairs, no running maximum (the reference moves
// only when a chunk's sum of P leaves [2^-64, 2^16], and the chunk is done again), stores of P straight
// to tensor memory.
//
// Measured: 4096 tokens of 32 heads of 32 on one axis 246 us, as bricks on three axes 431 us, eight frames of
// 1370 patches of 16 heads of 64 on two axes 250 us; 2.2 warp instructions a clock and SM, exponentials 25-40% of
// their rate, tensor pipe 12%.
//
// Tensor memory a tile, 128 columns: S [64 fp32] | P [32, bf16 pairs] | O [32] at d = 32; at d = 64 P lies
// over S (S 64 | O 64), is kept in registers until the chunk's sum has passed, and the next S waits for
// P V.  Either way four tiles are in flight an SM.
#include "relpos_tc.cuh"

namespace lsrm {
namespace rp {

template <int D>
struct TcFwd {
  static constexpr int kRowBytes = D * 2, kKeys = 64;
  static constexpr int kStages = D == 32 ? 4 : 3;
  static constexpr uint32_t kLayout = D == 32 ? kLayoutSW64 : kLayoutSW128;
  static constexpr uint32_t kAtomBytes = 8 * kRowBytes;
  static constexpr int kQBytes = 128 * kRowBytes, kKVBytes = kKeys * kRowBytes;
  static constexpr bool kAlias = D == 64;  // P over S
  static constexpr int kTileCols = 128, kTmemCols = 256;
  static constexpr int kColS = 0, kColP = kAlias ? 0 : 64, kColO = kAlias ? 64 : 96;
  static constexpr uint32_t kIdescQK = idesc_bf16(128, kKeys, false), kIdescPV = idesc_bf16(128, D, true);
  static_assert(kColO + D <= kTileCols, "tensor memory of a tile");
};

template <int D, int NA>
struct TcFwdSmem {
  using C = TcFwd<D>;
  uint8_t q[2][C::kQBytes];
  uint8_t k[C::kStages][C::kKVBytes];
  uint8_t v[C::kStages][C::kKVBytes];
  int pos[C::kStages][NA][C::kKeys];
  ChunkMeta meta[C::kStages];
  uint64_t q_full, kv_full[C::kStages], kv_empty[C::kStages], s_full[2], p_full[2], pv_done[2], drain;
  uint32_t tmem_base;
  int abort;
  float lut[1];  // [NA][2 maxd + 1]
  static size_t bytes(int maxd) { return sizeof(TcFwdSmem) + (size_t)NA * (2 * maxd + 1) * 4; }
};

template <int D, int NA>
__global__ void __launch_bounds__(kTcThreads, 2)
    rp_fwd_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const Params p) {
  using C = TcFwd<D>;
  using Smem = TcFwdSmem<D, NA>;
  // the operand tiles need 1024-byte alignment; an alignment computed here would cost the compiler the
  // address space, and with it the shared-memory forms of the table look-ups
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  if (smem_u32(smem_raw) & 1023) {
    raise_status(p.status, LSRM_ERR_CUDA);
    return;
  }

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_dependents();
  int unit = blockIdx.x;
  const int split = unit % p.splits;
  unit /= p.splits;
  const int h = unit % p.Hq, tile = unit / p.Hq, hk = h / p.G;
  int first, qlo, qhi, klo, khi;
  const int seg = seg_of_tile(p.off_q, p.S, p.Nq, 256, tile, first);
  seg_bounds(p.off_q, seg, p.Nq, qlo, qhi, p.status);
  const int row0 = qlo + (tile - first) * 256;
  if (tile < first || row0 >= qhi) return;
  seg_bounds(p.off_k, seg, p.Nk, klo, khi, p.status);
  const int nk = khi - klo, all = (nk + C::kKeys - 1) / C::kKeys;
  const int per = (all + p.splits - 1) / p.splits;
  const int c0 = min(split * per, all), chunks = min(c0 + per, all) - c0;
  const int k0 = klo + c0 * C::kKeys;  // first key of this CTA
  const int tiles = row0 + 128 < qhi ? 2 : 1, top = 2 * p.maxd;

  if (tid == 0) {
    S.abort = 0;
    mbar_init(&S.q_full, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&S.kv_full[s], 1);
      mbar_init(&S.kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&S.s_full[t], 1);
      mbar_init(&S.p_full[t], 128);
      mbar_init(&S.pv_done[t], 1);
    }
    mbar_init(&S.drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // The table in log2 units when every entry is small or -inf: the bias, the reference and the units then
  // fold into the exponent's multiply-add.  Otherwise in natural units, and the slow path (kFoldLimit).
  bool small = true;
  for (int i = tid; i <= top; i += kTcThreads) {
    const int b = checked_bucket(p, i);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const float x = b < 0 ? 0.0f : bf16_to_f32(p.table[((size_t)a * p.NB + b) * p.Hq + h]);
      small = small && (fabsf(x) <= kSmallBias || x == -INFINITY);
      S.lut[a * (top + 1) + i] = x;
    }
  }
  __syncwarp();
  tc_fence_before();
  const bool fold = __syncthreads_and(small);
  tc_fence_after();
  if (fold)  // every thread scales the entries that it wrote
    for (int i = tid; i <= top; i += kTcThreads)
#pragma unroll
      for (int a = 0; a < NA; ++a) S.lut[a * (top + 1) + i] *= kLog2e;
  __syncthreads();
  const float to_log2 = fold ? 1.0f : kLog2e;  // from the scores' units to log2
  const float mul = fold ? p.scale * kLog2e : p.scale;
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0 && chunks > 0) {
      mbar_arrive_expect_tx(&S.q_full, tiles * C::kQBytes);
      for (int t = 0; t < tiles; ++t) tma_load_3d(S.q[t], &qmap, &S.q_full, 0, h, row0 + t * 128);
    }
    int issued = 0;
    for (int c = 0; c < chunks; ++c) {
      const int st = c % C::kStages, key = k0 + c * C::kKeys, n = min(C::kKeys, khi - key);
      int x[NA][2];
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i)  // positions past the end repeat the last key's
          x[a][i] = p.pos_k[(size_t)(key + min(lane + 32 * i, n - 1)) * NA + a];
      if (c >= C::kStages && !wait_bar_w(&S.kv_empty[st], ((c / C::kStages) + 1) & 1, abort, p.status)) break;
      note_positions<NA>(x, S.pos[st], S.meta[st], lane, p.status);
      if (n < C::kKeys) {
        copy_tail<D>(S.v[st], p.v, key, n, p.Hkv, hk, lane);
        fence_async();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&S.kv_full[st], (n < C::kKeys ? 1 : 2) * C::kKVBytes);
        tma_load_3d(S.k[st], &kmap, &S.kv_full[st], 0, hk, key);
        if (n == C::kKeys) tma_load_3d(S.v[st], &vmap, &S.kv_full[st], 0, hk, key);
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
    // ---------------- MMA issuer: one thread, which mostly waits for the softmax ----------------
    if (lane == 0 && chunks > 0) {
      bool ok = wait_bar(&S.q_full, 0, abort, p.status);
      tc_fence_after();
      const uint64_t qdesc[2] = {smem_desc(smem_u32(S.q[0]), 16, C::kAtomBytes, C::kLayout),
                                 smem_desc(smem_u32(S.q[1]), 16, C::kAtomBytes, C::kLayout)};
      const uint64_t kdesc = smem_desc(smem_u32(S.k[0]), 16, C::kAtomBytes, C::kLayout);
      const uint64_t vdesc = smem_desc(smem_u32(S.v[0]), C::kKVBytes, C::kAtomBytes, C::kLayout);
      constexpr uint32_t kStep = C::kKVBytes >> 4;
      auto issue_qk = [&](int t, int c) {
        const uint32_t d = tmem + t * C::kTileCols + C::kColS;
        const uint64_t b = kdesc + (uint64_t)((c % C::kStages) * kStep);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) mma_ss(d, qdesc[t] + 2 * i, b + 2 * i, C::kIdescQK, i > 0 ? 1u : 0u);
        mma_commit(&S.s_full[t]);
      };
      auto issue_pv = [&](int t, int c) {
        const uint32_t d = tmem + t * C::kTileCols + C::kColO;
        const uint64_t b = vdesc + (uint64_t)((c % C::kStages) * kStep);
#pragma unroll
        for (int i = 0; i < C::kKeys / 16; ++i)
          mma_ts(d, tmem + t * C::kTileCols + C::kColP + i * 8, b + i * (16 * C::kRowBytes >> 4), C::kIdescPV,
                 (c == 0 && i == 0) ? 0u : 1u);
        mma_commit(&S.pv_done[t]);
      };
      for (int c = 0; ok && c < chunks; ++c) {
        if (!wait_bar(&S.kv_full[c % C::kStages], (c / C::kStages) & 1, abort, p.status)) { ok = false; break; }
        tc_fence_after();
        for (int t = 0; t < tiles; ++t) {
          if (c > 0) {
            if (!wait_bar(&S.p_full[t], (c - 1) & 1, abort, p.status)) { ok = false; break; }
            tc_fence_after();
          }
          if (!C::kAlias) {
            // S(c) ahead of P(c - 1) V: it overwrites only S, which the softmax released with P(c - 1)
            issue_qk(t, c);
            if (c > 0) issue_pv(t, c - 1);
          } else if (c > 0) {
            issue_pv(t, c - 1);
          }
        }
        if (!ok) break;
        if (C::kAlias) {
          for (int t = 0; t < tiles; ++t) {
            // S(c) overwrites P(c - 1), so that product has to be done
            if (c > 0 && !wait_bar(&S.pv_done[t], (c - 1) & 1, abort, p.status)) { ok = false; break; }
            tc_fence_after();
            issue_qk(t, c);
          }
          if (!ok) break;
        }
        if (c > 0) mma_commit(&S.kv_empty[(c - 1) % C::kStages]);
      }
      for (int t = 0; ok && t < tiles; ++t) {
        if (!wait_bar(&S.p_full[t], (chunks - 1) & 1, abort, p.status)) { ok = false; break; }
        tc_fence_after();
        issue_pv(t, chunks - 1);
      }
      // every MMA issued so far must finish before the CTA can release tensor and shared memory
      mma_commit(&S.drain);
      volatile int no_abort = 0;
      wait_bar(&S.drain, 0, &no_abort, nullptr);
    }
  } else if (((warp - 2) >> 2) < tiles) {
    // ---------------- softmax: one row a thread ----------------
    const int t = (warp - 2) >> 2, quarter = warp & 3;  // tensor-memory lanes this warp may access
    const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16) + t * C::kTileCols;
    const int row = row0 + t * 128 + quarter * 32 + lane;
    const bool valid = row < qhi;
    int rowc[NA], q_lo[NA], q_hi[NA];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int x = p.pos_q[(size_t)min(row, qhi - 1) * NA + a];
      rowc[a] = p.maxd - x;
      q_lo[a] = __reduce_min_sync(0xffffffffu, x);
      q_hi[a] = __reduce_max_sync(0xffffffffu, x);
      if (q_lo[a] < -kPosLimit || q_hi[a] > kPosLimit) raise_status(p.status, LSRM_ERR_BOUNDS);
    }
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool { return wait_bar_w(bar, parity, abort, p.status); };

    float m = 0.0f, l = 0.0f;  // the row's reference (in the scores' units) and sum
    bool ok = true;
    int st = 0, left = 0;  // the current chunk's stage and keys from here on
    ChunkBias<NA> cb;

    // The chunk again, or a chunk of a table too large to fold: its maximum, the reference of the rows
    // that are `off` (or, without folding, behind their maximum) moved to it, and P from the scores in
    // the formula's order.  Returns the row's sum.
    auto slow_chunk = [&](int c, bool off) -> float {
      float mx = -INFINITY, sum = 0.0f;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t r[16];
        float b[16];
        tmem_ld16(tbase + C::kColS + 16 * g, r);
        tmem_wait16(r);
        cb.exact16(b, r, mul, S.pos[st], g, rowc, S.lut, top);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (16 * g + e < left) mx = fmaxf(mx, b[e]);
      }
      if (!fold) off = valid && (c == 0 || mx > m);
      const float f = !off ? 1.0f : m == -INFINITY ? 0.0f : ex2((m - mx) * to_log2);
      if (c > 0 && __any_sync(0xffffffffu, off)) {
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(tbase + C::kColO + 32 * i, o);
          tmem_wait32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st32(tbase + C::kColO + 32 * i, o);
        }
        l *= f;
      }
      if (off) m = mx;
      const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        uint32_t r[16], pk[8];
        float b[16];
        tmem_ld16(tbase + C::kColS + 16 * g, r);
        tmem_wait16(r);
        cb.exact16(b, r, mul, S.pos[st], g, rowc, S.lut, top);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = ex2((b[e] - ref) * to_log2);
          b[e] = 16 * g + e < left ? x : 0.0f;
          sum += b[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = pack2(b[2 * e], b[2 * e + 1]);
        tmem_st8(tbase + C::kColP + 8 * g, pk);  // over S only where it has been read
      }
      return sum;
    };

    for (int c = 0; c < chunks; ++c) {
      st = c % C::kStages;
      left = khi - k0 - c * C::kKeys;
      if (!wait_all(&S.kv_full[st], (c / C::kStages) & 1) || !wait_all(&S.s_full[t], c & 1)) { ok = false; break; }
      tc_fence_after();
      cb.set(S.meta[st], q_lo, q_hi, p.maxd, S.lut, top);
      if (!C::kAlias && c > 0 && !wait_all(&S.pv_done[t], (c - 1) & 1)) { ok = false; break; }  // P is free
      tc_fence_after();
      float sum;
      if (!fold) {
        sum = slow_chunk(c, false);
      } else {
        const float base = cb.ub - (m == -INFINITY ? 0.0f : m);
        uint32_t pk[C::kAlias ? 32 : 16];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll(C::kAlias ? 2 : 1)
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t r[32];
          tmem_ld32(tbase + C::kColS + 32 * hf, r);
          tmem_wait32(r);
          uint32_t* to = C::kAlias ? pk + 16 * hf : pk;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float b[16];
            const float one = cb.row16(base, S.pos[st], 2 * hf + g, rowc, S.lut, top);
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              ffma2(b[e], b[e + 1], __uint_as_float(r[16 * g + e]), __uint_as_float(r[16 * g + e + 1]), mul, one);
            if (!cb.flat(2 * hf + g)) cb.add16(b, S.pos[st], 2 * hf + g, rowc, S.lut, top);
            if (left < 32 * hf + 16 * g + 16) {
              keep_branch();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (32 * hf + 16 * g + e >= left) b[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float p0 = ex2(b[e]), p1 = ex2(b[e + 1]);
              fadd2_acc(s0, s1, p0, p1);
              to[8 * g + e / 2] = pack2(p0, p1);
            }
          }
          if (!C::kAlias) tmem_st16(tbase + C::kColP + 16 * hf, pk);
        }
        sum = s0 + s1;
        const bool off = valid && (c == 0 ? !(sum <= 65536.0f && sum >= 5.421010862427522e-20f)
                                          : !(sum <= 65536.0f) || m == -INFINITY);
        if (__any_sync(0xffffffffu, off)) {
          sum = slow_chunk(c, off);
        } else if (C::kAlias) {
          tmem_st32(tbase + C::kColP, pk);
        }
      }
      l += sum;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&S.p_full[t]);
    }
    if (ok && chunks > 0) ok = wait_all(&S.pv_done[t], (chunks - 1) & 1);
    tc_fence_after();
    if (ok) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const size_t at = (size_t)row * p.Hq + h;
      const size_t pat = (size_t)split * p.Nq * p.Hq + at;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (chunks > 0) {
          tmem_ld32(tbase + C::kColO + 32 * i, o);
          tmem_wait32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (!valid) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
        if (p.splits == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + 32 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* x = reinterpret_cast<const float*>(o + 8 * e);
            dst[e] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]),
                                pack2(x[6], x[7]));
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.o_part + pat * D + 32 * i);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (valid) {
        if (p.splits > 1)
          p.ml_part[pat] = make_float2(l == 0.0f ? -INFINITY : fold ? m * kLn2 : m, l);
        else if (p.lse != nullptr)
          p.lse[at] = l == 0.0f ? -INFINITY : (fold ? m * kLn2 : m) + logf(l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int NA>
static lsrm_status run_tc(const Params& p, long long ctas, cudaStream_t s) {
  CUtensorMap qm, km, vm;
  // without a key no copy is made, but a map needs a tensor
  const bool keys = p.Nk > 0;
  if (!make_map(&qm, p.q, D, p.Hq, p.Nq, 1, 128) ||
      !make_map(&km, keys ? p.k : p.q, D, keys ? p.Hkv : p.Hq, keys ? p.Nk : p.Nq, 1, 64) ||
      !make_map(&vm, keys ? p.v : p.q, D, keys ? p.Hkv : p.Hq, keys ? p.Nk : p.Nq, 1, 64))
    return LSRM_ERR_CUDA;
  const size_t bytes = TcFwdSmem<D, NA>::bytes(p.maxd);
  if (!allow_smem(rp_fwd_tc_kernel<D, NA>, bytes)) return LSRM_ERR_CUDA;
  rp_fwd_tc_kernel<D, NA><<<(unsigned)ctas, kTcThreads, bytes, s>>>(qm, km, vm, p);
  return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

lsrm_status launch_fwd_tc(const Params& p, int D, int NA, long long ctas, cudaStream_t s) {
  if (D == 32)
    return NA == 1 ? run_tc<32, 1>(p, ctas, s) : NA == 2 ? run_tc<32, 2>(p, ctas, s) : run_tc<32, 3>(p, ctas, s);
  return NA == 1 ? run_tc<64, 1>(p, ctas, s) : NA == 2 ? run_tc<64, 2>(p, ctas, s) : run_tc<64, 3>(p, ctas, s);
}

}  // namespace rp
}  // namespace lsrm
