// Layer norm of rows, forward and backward, with the reduction of the weights' gradients.
//
//   mean = sum(x) / C,  rstd = 1 / sqrt(sum((x - mean)^2) / C + eps),  xh = (x - mean) rstd
//   y = xh gamma + beta
//   g = dy gamma,  dx = rstd (g - mean(g) - xh mean(g xh)),  dgamma = sum_rows dy xh,
//   dbeta = sum_rows dy
//
// Both directions are bound by HBM: the forward reads x and writes y, the backward reads x and dy
// and writes dx, once each.  So a row lives in the registers of the lanes that share it (a group of
// 1..32 lanes of a warp, or a whole CTA for wide rows) between its statistics and its output, and
// the variance is the two-pass one (deviations from the row's own mean), which needs no second read.
// Rows too wide for registers are read again from the caches.
//
// The backward keeps the column sums of dgamma and dbeta in registers over all rows a thread meets
// (a grid of as many CTAs as are resident, each walking its rows), adds the CTA's partials in
// shared memory in a fixed order, and a second kernel adds the CTAs' partials in a fixed order: no
// float atomics, so the gradients are the same bit for bit on every run.  All sums are fp32.
#include <climits>
#include <type_traits>

#include "lsrm_common.cuh"

namespace lsrm {
namespace {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;
constexpr int kLnSms = 148;
constexpr int kLnWidest = 8192;  // elements of a row that the backward keeps in registers, at most
constexpr int kLnWideSplits = 64;

// ---- element types ----
template <typename T>
__device__ __forceinline__ float ln_to_f32(T v);
template <>
__device__ __forceinline__ float ln_to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float ln_to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <typename T>
__device__ __forceinline__ T ln_from_f32(float v);
template <>
__device__ __forceinline__ float ln_from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t ln_from_f32<uint16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// VEC consecutive elements as loaded: 16 bytes, or one element where the rows are not aligned.
// Plain (coherent) loads: y may be x, and dx may be dy or x.
template <typename T, int VEC>
struct LnVec {
  static_assert(VEC == 1 || VEC * sizeof(T) == 16, "16-byte vectors or single elements");
  T v[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1) {
      v[0] = *p;
    } else {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == 1) {
      *p = v[0];
    } else {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = T(0);
  }
  __device__ __forceinline__ float get(int e) const { return ln_to_f32<T>(v[e]); }
  __device__ __forceinline__ void set(int e, float f) { v[e] = ln_from_f32<T>(f); }
};

// sum over the TPR threads that share a row: a lane group of a warp, or the whole CTA
template <int TPR>
__device__ __forceinline__ float ln_row_sum(float v, float* red) {
  constexpr int kLanes = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    static_assert(TPR == kLnThreads, "a row belongs to a lane group or to the CTA");
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLnWarps; ++w) v += red[w];
  }
  return v;
}

struct LnFwd {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  long long rows;
  int C;
  float eps;
};

// Rows in registers: TPR threads a row, NV vectors of VEC elements a thread (C <= TPR * VEC * NV)
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kLnThreads) ln_fwd_kernel(const LnFwd p) {
  __shared__ float red[kLnWarps];
  constexpr int kRowsPerCta = kLnThreads / TPR;
  const int sub = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * kRowsPerCta + threadIdx.x / TPR;
  const bool live = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.C;
  LnVec<T, VEC> xv[NV];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + sub) * VEC;
    if (live && c < p.C)
      xv[i].load(x + c);
    else
      xv[i].zero();
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += xv[i].get(e);
  const float mean = ln_row_sum<TPR>(s, red) / (float)p.C;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * TPR + sub) * VEC < p.C) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = xv[i].get(e) - mean;
        s = fmaf(d, d, s);
      }
    }
  }
  const float rstd = rsqrtf(ln_row_sum<TPR>(s, red) / (float)p.C + p.eps);
  if (!live) return;
  T* y = static_cast<T*>(p.y) + row * p.C;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + sub) * VEC;
    if (c >= p.C) continue;
    LnVec<T, VEC> gv, bv;
    if (p.gamma != nullptr) gv.load(static_cast<const T*>(p.gamma) + c);
    if (p.beta != nullptr) bv.load(static_cast<const T*>(p.beta) + c);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float o = (xv[i].get(e) - mean) * rstd;
      if (p.gamma != nullptr) o *= gv.get(e);
      if (p.beta != nullptr) o += bv.get(e);
      xv[i].set(e, o);
    }
    xv[i].store(y + c);
  }
  if (sub == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

// Rows of any width, one CTA each, read three times (the later reads come from the caches)
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_fwd_wide_kernel(const LnFwd p) {
  __shared__ float red[kLnWarps];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.C;
  T* y = static_cast<T*>(p.y) + row * p.C;
  const T* gamma = static_cast<const T*>(p.gamma);
  const T* beta = static_cast<const T*>(p.beta);
  float s = 0.0f;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) s += ln_to_f32<T>(x[c]);
  const float mean = ln_row_sum<kLnThreads>(s, red) / (float)p.C;
  s = 0.0f;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    const float d = ln_to_f32<T>(x[c]) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = rsqrtf(ln_row_sum<kLnThreads>(s, red) / (float)p.C + p.eps);
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    float o = (ln_to_f32<T>(x[c]) - mean) * rstd;
    if (gamma != nullptr) o *= ln_to_f32<T>(gamma[c]);
    if (beta != nullptr) o += ln_to_f32<T>(beta[c]);
    y[c] = ln_from_f32<T>(o);
  }
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
}

struct LnBwd {
  const void* dy;
  const void* x;
  const void* gamma;
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;  // [CTAs][2][C]: the CTA's sums of dgamma and dbeta
  long long rows;
  int C;
};

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_kernel(const LnBwd p) {
  __shared__ float red[kLnWarps];
  __shared__ float cols[TPR < kLnThreads ? kLnWarps : 1][2][TPR < kLnThreads ? 32 * VEC : 1];
  constexpr int kRowsPerCta = kLnThreads / TPR;
  const int sub = threadIdx.x % TPR;
  LnVec<T, VEC> gv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + sub) * VEC;
    gv[i].zero();
    if (c < p.C) {
      if (p.gamma != nullptr)
        gv[i].load(static_cast<const T*>(p.gamma) + c);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) gv[i].set(e, 1.0f);
    }
  }
  float dg[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dg[i][e] = db[i][e] = 0.0f;

  const float inv_c = 1.0f / (float)p.C;
  const long long steps = (p.rows + kRowsPerCta - 1) / kRowsPerCta;
  for (long long it = blockIdx.x; it < steps; it += gridDim.x) {
    const long long row = it * kRowsPerCta + threadIdx.x / TPR;
    const bool live = row < p.rows;
    const long long at = (live ? row : 0) * p.C;
    const float mean = live ? p.mean[row] : 0.0f, rstd = live ? p.rstd[row] : 0.0f;
    LnVec<T, VEC> xv[NV], dv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + sub) * VEC;
      if (live && c < p.C) {
        xv[i].load(static_cast<const T*>(p.x) + at + c);
        dv[i].load(static_cast<const T*>(p.dy) + at + c);
      } else {
        xv[i].zero();
        dv[i].zero();
      }
    }
    float sg = 0.0f, sgx = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xh = (xv[i].get(e) - mean) * rstd, d = dv[i].get(e), g = d * gv[i].get(e);
        sg += g;
        sgx = fmaf(g, xh, sgx);
        dg[i][e] = fmaf(d, xh, dg[i][e]);
        db[i][e] += d;
      }
    sg = ln_row_sum<TPR>(sg, red) * inv_c;
    sgx = ln_row_sum<TPR>(sgx, red) * inv_c;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + sub) * VEC;
        if (c >= p.C) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (xv[i].get(e) - mean) * rstd, g = dv[i].get(e) * gv[i].get(e);
          xv[i].set(e, rstd * (g - sg - xh * sgx));
        }
        xv[i].store(static_cast<T*>(p.dx) + at + c);
      }
    }
  }

  // the CTA's column sums, in a fixed order
  float* part = p.part + (long long)blockIdx.x * 2 * p.C;
  if constexpr (TPR == kLnThreads) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + sub) * VEC;
      if (c >= p.C) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        part[c + e] = dg[i][e];
        part[p.C + c + e] = db[i][e];
      }
    }
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float a = dg[i][e], b = db[i][e];
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (lane < TPR) {
          cols[warp][0][lane * VEC + e] = a;
          cols[warp][1][lane * VEC + e] = b;
        }
      }
      __syncthreads();
      for (int t = threadIdx.x; t < 2 * TPR * VEC; t += kLnThreads) {
        const int which = t / (TPR * VEC), c = t % (TPR * VEC), col = i * TPR * VEC + c;
        if (col >= p.C) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kLnWarps; ++w) s += cols[w][which][c];
        part[which * p.C + col] = s;
      }
    }
  }
}

// dx of rows of any width (one CTA each, two reads); the weights' sums come from ln_bwd_cols_kernel
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_wide_kernel(const LnBwd p) {
  __shared__ float red[kLnWarps];
  const long long row = blockIdx.x, at = row * p.C;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* dy = static_cast<const T*>(p.dy) + at;
  const T* gamma = static_cast<const T*>(p.gamma);
  T* dx = static_cast<T*>(p.dx) + at;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float sg = 0.0f, sgx = 0.0f;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    const float g = ln_to_f32<T>(dy[c]) * (gamma != nullptr ? ln_to_f32<T>(gamma[c]) : 1.0f);
    sg += g;
    sgx = fmaf(g, (ln_to_f32<T>(x[c]) - mean) * rstd, sgx);
  }
  sg = ln_row_sum<kLnThreads>(sg, red) / (float)p.C;
  sgx = ln_row_sum<kLnThreads>(sgx, red) / (float)p.C;
  for (int c = threadIdx.x; c < p.C; c += kLnThreads) {
    const float g = ln_to_f32<T>(dy[c]) * (gamma != nullptr ? ln_to_f32<T>(gamma[c]) : 1.0f);
    dx[c] = ln_from_f32<T>(rstd * (g - sg - (ln_to_f32<T>(x[c]) - mean) * rstd * sgx));
  }
}

// column sums of a run of rows (grid: column tiles x row splits), before dx may overwrite x or dy
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_cols_kernel(const LnBwd p) {
  const int c = blockIdx.x * kLnThreads + threadIdx.x;
  if (c >= p.C) return;
  const long long per = (p.rows + gridDim.y - 1) / gridDim.y;
  const long long r0 = blockIdx.y * per, r1 = min(r0 + per, p.rows);
  float a = 0.0f, b = 0.0f;
  for (long long r = r0; r < r1; ++r) {
    const float d = ln_to_f32<T>(static_cast<const T*>(p.dy)[r * p.C + c]);
    const float xh = (ln_to_f32<T>(static_cast<const T*>(p.x)[r * p.C + c]) - p.mean[r]) * p.rstd[r];
    a = fmaf(d, xh, a);
    b += d;
  }
  float* part = p.part + (long long)blockIdx.y * 2 * p.C;
  part[c] = a;
  part[p.C + c] = b;
}

// dgamma / dbeta = the sum of the CTAs' partials: 32 columns a CTA, its warps take every
// kLnWarps-th partial, and the warps' sums are added in order
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_bwd_finish_kernel(const float* part, int n, int C, void* dgamma,
                                                                   void* dbeta) {
  __shared__ float s[2][kLnWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.0f, b = 0.0f;
  if (c < C) {
    for (int i = warp; i < n; i += kLnWarps) {
      a += part[(long long)i * 2 * C + c];
      b += part[(long long)i * 2 * C + C + c];
    }
  }
  s[0][warp][lane] = a;
  s[1][warp][lane] = b;
  __syncthreads();
  if (warp >= 2 || c >= C) return;
  void* out = warp == 0 ? dgamma : dbeta;
  if (out == nullptr) return;
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kLnWarps; ++w) t += s[warp][w][lane];
  static_cast<T*>(out)[c] = ln_from_f32<T>(t);
}

// ---- variants: by the row's width, the element type and alignment alone ----
//
// Aligned rows (C a multiple of the vector, pointers on 16 bytes): the fewest lanes that hold the
// row with one vector each up to a warp, then up to kNvMax vectors a lane, then a CTA a row.
// Others: single elements, coalesced across the lanes.
struct LnShape {
  int vec, tpr, nv;  // nv = 0: the wide kernels
};

LnShape ln_shape(int C, int elem, bool vec_ok, bool backward) {
  const int vec = vec_ok ? 16 / elem : 1;
  const int n = (C + vec - 1) / vec;  // vectors a row
  // elements a lane may hold: the backward keeps two fp32 sums per element beside the row itself
  const int most = vec_ok ? (backward ? 32 / vec : 64 / vec) : (backward ? 16 : 32);
  int tpr = 1;
  while (tpr < 32 && tpr < n) tpr *= 2;
  int nv = 1;
  while (nv * tpr < n) nv *= 2;
  if (nv <= most) return {vec, tpr, nv};
  tpr = kLnThreads;
  nv = 1;
  while (nv * tpr < n) nv *= 2;
  if (nv <= most) return {vec, tpr, nv};
  return {1, kLnThreads, 0};
}

template <typename T, int VEC, int TPR, int NV>
lsrm_status ln_run_fwd(const LnFwd& p, cudaStream_t s) {
  constexpr int kRows = kLnThreads / TPR;
  const long long ctas = (p.rows + kRows - 1) / kRows;
  if (ctas > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
  ln_fwd_kernel<T, VEC, TPR, NV><<<(unsigned)ctas, kLnThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

template <typename T, int VEC, int TPR, int NV>
lsrm_status ln_run_bwd(const LnBwd& p, int max_ctas, int* ctas, cudaStream_t s) {
  constexpr int kRows = kLnThreads / TPR;
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, ln_bwd_kernel<T, VEC, TPR, NV>, kLnThreads, 0) !=
      cudaSuccess)
    return LSRM_ERR_CUDA;
  const long long want = (p.rows + kRows - 1) / kRows, fit = (long long)kLnSms * (per_sm > 0 ? per_sm : 1);
  long long n = want < fit ? want : fit;
  if (n > max_ctas) n = max_ctas;
  if (n < 1) return LSRM_ERR_CUDA;
  *ctas = (int)n;
  ln_bwd_kernel<T, VEC, TPR, NV><<<(unsigned)n, kLnThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

// f(vector width, threads a row, vectors a thread) with the shape as template arguments
template <int V, int N>
struct LnTag {
  static constexpr int vec = V, nv = N;
};
template <int TPR, typename T, typename F>
lsrm_status ln_nv(const LnShape& h, F f) {
  constexpr int V = 16 / sizeof(T);
  if (h.vec == V) {
    switch (h.nv) {
      case 1: return f(LnTag<V, 1>{}, std::integral_constant<int, TPR>{});
      case 2: if constexpr (TPR >= 32) return f(LnTag<V, 2>{}, std::integral_constant<int, TPR>{}); break;
      case 4: if constexpr (TPR >= 32) return f(LnTag<V, 4>{}, std::integral_constant<int, TPR>{}); break;
      case 8: if constexpr (TPR >= 32) return f(LnTag<V, 8>{}, std::integral_constant<int, TPR>{}); break;
      case 16: if constexpr (TPR >= 32 && V == 4) return f(LnTag<V, 16>{}, std::integral_constant<int, TPR>{}); break;
    }
  } else {
    switch (h.nv) {
      case 1: return f(LnTag<1, 1>{}, std::integral_constant<int, TPR>{});
      case 2: if constexpr (TPR >= 32) return f(LnTag<1, 2>{}, std::integral_constant<int, TPR>{}); break;
      case 4: if constexpr (TPR >= 32) return f(LnTag<1, 4>{}, std::integral_constant<int, TPR>{}); break;
      case 8: if constexpr (TPR >= 32) return f(LnTag<1, 8>{}, std::integral_constant<int, TPR>{}); break;
      case 16: if constexpr (TPR >= 32) return f(LnTag<1, 16>{}, std::integral_constant<int, TPR>{}); break;
      case 32: if constexpr (TPR >= 32) return f(LnTag<1, 32>{}, std::integral_constant<int, TPR>{}); break;
    }
  }
  return LSRM_ERR_UNSUPPORTED;
}
template <typename T, typename F>
lsrm_status ln_dispatch(const LnShape& h, F f) {
  switch (h.tpr) {
    case 1: return ln_nv<1, T>(h, f);
    case 2: return ln_nv<2, T>(h, f);
    case 4: return ln_nv<4, T>(h, f);
    case 8: return ln_nv<8, T>(h, f);
    case 16: return ln_nv<16, T>(h, f);
    case 32: return ln_nv<32, T>(h, f);
    case kLnThreads: return ln_nv<kLnThreads, T>(h, f);
  }
  return LSRM_ERR_UNSUPPORTED;
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename T>
lsrm_status ln_forward(const LnFwd& p, cudaStream_t s) {
  const bool vec_ok = (p.C * sizeof(T)) % 16 == 0 && on16(p.x) && on16(p.y) && on16(p.gamma) && on16(p.beta);
  const LnShape h = ln_shape(p.C, (int)sizeof(T), vec_ok, false);
  if (h.nv == 0) {
    if (p.rows > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
    ln_fwd_wide_kernel<T><<<(unsigned)p.rows, kLnThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
  }
  return ln_dispatch<T>(h, [&](auto tag, auto tpr) {
    return ln_run_fwd<T, decltype(tag)::vec, decltype(tpr)::value, decltype(tag)::nv>(p, s);
  });
}

template <typename T>
lsrm_status ln_backward(const LnBwd& p, void* dgamma, void* dbeta, int max_ctas, cudaStream_t s) {
  const bool vec_ok = (p.C * sizeof(T)) % 16 == 0 && on16(p.x) && on16(p.dy) && on16(p.dx) && on16(p.gamma);
  const LnShape h = ln_shape(p.C, (int)sizeof(T), vec_ok, true);
  int n = 0;
  if (p.rows > 0) {
    if (h.nv == 0) {
      if (p.rows > (long long)INT32_MAX) return LSRM_ERR_UNSUPPORTED;
      n = (int)(p.rows < kLnWideSplits ? p.rows : kLnWideSplits);
      if (n > max_ctas) n = max_ctas;
      const dim3 grid((unsigned)((p.C + kLnThreads - 1) / kLnThreads), (unsigned)n);
      ln_bwd_cols_kernel<T><<<grid, kLnThreads, 0, s>>>(p);
      if (cudaGetLastError() != cudaSuccess) return LSRM_ERR_CUDA;
      ln_bwd_wide_kernel<T><<<(unsigned)p.rows, kLnThreads, 0, s>>>(p);
      if (cudaGetLastError() != cudaSuccess) return LSRM_ERR_CUDA;
    } else {
      const lsrm_status st = ln_dispatch<T>(h, [&](auto tag, auto tpr) {
        return ln_run_bwd<T, decltype(tag)::vec, decltype(tpr)::value, decltype(tag)::nv>(p, max_ctas, &n, s);
      });
      if (st != LSRM_OK) return st;
    }
  }
  if (dgamma == nullptr && dbeta == nullptr) return LSRM_OK;
  ln_bwd_finish_kernel<T><<<(unsigned)((p.C + 31) / 32), kLnThreads, 0, s>>>(p.part, n, p.C, dgamma, dbeta);
  return cudaGetLastError() == cudaSuccess ? LSRM_OK : LSRM_ERR_CUDA;
}

}  // namespace

// CTAs whose partial sums the workspace holds: as many as can be resident (8 of 256 threads an SM),
// or one a row where there are fewer rows.  Rows above kLnWidest never fit registers; their column
// sums are split kLnWideSplits ways.
int ln_max_ctas(long long rows, int C) {
  const long long most = C > kLnWidest ? kLnWideSplits : 8 * kLnSms;
  return (int)(rows < most ? (rows > 0 ? rows : 1) : most);
}

lsrm_status launch_layer_norm_forward(long long rows, int C, int dtype, const void* x, const void* gamma,
                                      const void* beta, float eps, void* y, float* mean, float* rstd,
                                      cudaStream_t s) {
  const LnFwd p{x, gamma, beta, y, mean, rstd, rows, C, eps};
  return dtype == LSRM_F32 ? ln_forward<float>(p, s) : ln_forward<uint16_t>(p, s);
}

lsrm_status launch_layer_norm_backward(long long rows, int C, int dtype, const void* dy, const void* x,
                                       const void* gamma, const float* mean, const float* rstd, void* dx,
                                       void* dgamma, void* dbeta, float* part, cudaStream_t s) {
  const LnBwd p{dy, x, gamma, mean, rstd, dx, part, rows, C};
  const int most = ln_max_ctas(rows, C);
  return dtype == LSRM_F32 ? ln_backward<float>(p, dgamma, dbeta, most, s)
                           : ln_backward<uint16_t>(p, dgamma, dbeta, most, s);
}

}  // namespace lsrm
